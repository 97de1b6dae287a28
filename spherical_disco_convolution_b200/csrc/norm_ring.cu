// Layer norm over channels for long planes: the tiles of x (and dout) pass through a ring in
// shared memory.  Formulas and sums as in norm.cu.
//
// What bounds both passes is HBM, and what kept the register form below it was latency: its
// loads are only in flight between two barriers of a CTA.  Here the ring is kept full of
// tiles of C channels x LPR * VEC points (one TMA box, or one bulk copy per channel row where
// rows do not start on 16 bytes) while two groups of eight warps take tiles in turn, so that one
// group computes while the other waits at its barriers.  A tile is read from HBM once and from
// shared memory twice, for the sums and for the result.  LPR = 32 or 16 lanes take a channel
// row, VEC points each (16 warps and none besides leave a thread 128 registers: the first warp of
// the group that has done with a tile loads the next one into its place), so a group has 8 or 16 rows of lanes and row r takes the channels r,
// r + rows, ...; the sums over channels cross the rows through shared memory.
//
// Forward sums in one pass: a row of lanes adds v = x - k and v^2 about the value k of its first
// channel.  k is one of the n values it adds, so (mean - k)^2 is at most n times their variance and
// m2 = sum v^2 - (sum v)^2 / n loses at most log2(n) + 1 bits; the rows then combine as in norm.cu.
//
// Rows that do not start on 16 bytes: the copy takes every 16-byte block that holds a value of
// the row's piece, and the row is read from its own offset, one element at a time.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "common.cuh"
#include "kernels.h"
#include "norm.h"
#include "tc_common.cuh"

namespace disco {
namespace {

constexpr int kWarps = 8;                     // of a group
constexpr int kGroup = kWarps * 32;
constexpr int kGroups = 2;
constexpr int kThreads = kGroups * kGroup;
constexpr int kMaxStages = 8;
constexpr size_t kRingSmem = 225 * 1024;      // of 227 KB

// Two fp32 values in one 64-bit register pair (sm_100's packed fp32 arithmetic).
struct F2 {
  unsigned long long v;
};
__device__ __forceinline__ F2 pack(float a, float b) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 unpack(F2 a) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a.v));
  return r;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}
__device__ __forceinline__ F2 neg2(F2 a) { return F2{a.v ^ 0x8000000080000000ull}; }

struct RingArgs {
  int B, C;
  int npts;
  int tiles_per_plane;
  long long tiles;
  int stages, stage_bytes;
  int dout_off, stat_off;      // byte offsets in a stage: dout rows, statistics rows
  int boxes, box_rows;         // TMA boxes per array
  const void* x;
  const void* dout;
  const float* stats_in;
  const void* gain;
  const void* bias;
  float eps;
  void* out;                   // forward: out, backward: dx (may be null)
  float* stats;
  float* part;
};

// A lane's points of one channel row, as VEC / 2 pairs (VEC = 1: one pair, its upper half 0).
// SHIFT rows hold point lane + LPR e in element e, others VEC consecutive points.
template <typename T, int VEC, int LPR, bool SHIFT>
__device__ __forceinline__ void read_row(const uint8_t* row, int lane, F2 (&v)[(VEC + 1) / 2]) {
  constexpr int kBytes = VEC * (int)sizeof(T);
  if constexpr (SHIFT || VEC == 1) {
    const T* p = reinterpret_cast<const T*>(row) + lane;
    float f[VEC + 1];
    f[VEC] = 0.0f;
#pragma unroll
    for (int e = 0; e < VEC; ++e) f[e] = to_f32(p[LPR * e]);
#pragma unroll
    for (int k = 0; k < (VEC + 1) / 2; ++k) v[k] = pack(f[2 * k], f[2 * k + 1]);
  } else {
    const uint8_t* p = row + lane * kBytes;
    uint32_t w[kBytes / 4];
    if constexpr (kBytes == 4) w[0] = *reinterpret_cast<const uint32_t*>(p);
    else if constexpr (kBytes == 8) {
      const uint2 q = *reinterpret_cast<const uint2*>(p);
      w[0] = q.x;
      w[1] = q.y;
    } else {
      const uint4 q = *reinterpret_cast<const uint4*>(p);
      w[0] = q.x;
      w[1] = q.y;
      w[2] = q.z;
      w[3] = q.w;
    }
#pragma unroll
    for (int k = 0; k < VEC / 2; ++k) {
      if constexpr (sizeof(T) == 2) v[k] = pack(__uint_as_float(w[k] << 16), __uint_as_float(w[k] & 0xffff0000u));
      else v[k] = pack(__uint_as_float(w[2 * k]), __uint_as_float(w[2 * k + 1]));
    }
  }
}

template <typename T, int VEC, int LPR, bool SHIFT>
__device__ __forceinline__ void write_row(T* dst, int lane, int valid, const F2 (&v)[(VEC + 1) / 2]) {
  constexpr int kBytes = VEC * (int)sizeof(T);
  float f[VEC + 1];
#pragma unroll
  for (int k = 0; k < (VEC + 1) / 2; ++k) {
    const float2 q = unpack(v[k]);
    f[2 * k] = q.x;
    f[2 * k + 1] = q.y;
  }
  if constexpr (SHIFT || VEC == 1) {
#pragma unroll
    for (int e = 0; e < VEC; ++e)
      if (lane + LPR * e < valid) dst[lane + LPR * e] = from_f32<T>(f[e]);
  } else {
    if (lane * VEC >= valid) return;
    uint32_t w[kBytes / 4];
#pragma unroll
    for (int k = 0; k < kBytes / 4; ++k) {
      if constexpr (sizeof(T) == 2) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * k], f[2 * k + 1]);
        w[k] = *reinterpret_cast<const uint32_t*>(&h);
      } else {
        w[k] = __float_as_uint(f[k]);
      }
    }
    T* p = dst + lane * VEC;
    if constexpr (kBytes == 4) *reinterpret_cast<uint32_t*>(p) = w[0];
    else if constexpr (kBytes == 8) *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
    else *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

template <typename T, int PTS, bool SHIFT>
constexpr int kPitch = PTS * (int)sizeof(T) + (SHIFT ? 16 : 0);
template <int PTS, bool SHIFT>
constexpr int kStatPitch = PTS * 4 + (SHIFT ? 16 : 0);

// Bytes by which element `at` of an array at `base` lies past a 16-byte boundary.
template <typename T>
__device__ __forceinline__ uint32_t past16(const T* base, size_t at) {
  return (uint32_t)(reinterpret_cast<uintptr_t>(base + at) & 15);
}

struct Ring {
  uint8_t* stage;
  uint64_t* full;
  uint64_t* empty;
};

// One warp: tile k of this CTA into stage k % stages, which is free.
template <typename T, int kPts, bool SHIFT, bool BWD>
__device__ __forceinline__ void load_tile(const RingArgs& a, const CUtensorMap* map_x, const CUtensorMap* map_d,
                                          const Ring& r, int k) {
  const long long tile = blockIdx.x + (long long)k * gridDim.x;
  if (tile >= a.tiles) return;
  const int lane = threadIdx.x & 31, st = k % a.stages;
  const int b = (int)(tile / a.tiles_per_plane), p0 = (int)(tile % a.tiles_per_plane) * kPts;
  const int valid = min(kPts, a.npts - p0);
  uint8_t* base = r.stage + (size_t)st * a.stage_bytes;
  if constexpr (!SHIFT) {
    if (lane == 0) {
      const uint32_t rows = (uint32_t)(a.boxes * a.box_rows * kPitch<T, kPts, SHIFT>);
      tc::mbar_arrive_expect_tx(&r.full[st], BWD ? 2 * rows + 8u * valid : rows);
      for (int i = 0; i < a.boxes; ++i) {
        tc::tma_load_3d(base + i * a.box_rows * kPitch<T, kPts, SHIFT>, map_x, &r.full[st], p0, i * a.box_rows, b);
        if (BWD)
          tc::tma_load_3d(base + a.dout_off + i * a.box_rows * kPitch<T, kPts, SHIFT>, map_d, &r.full[st], p0,
                          i * a.box_rows, b);
      }
      if (BWD) {
        const float* s = a.stats_in + (size_t)b * a.npts + p0;
        tc::bulk_load(base + a.stat_off, s, 4 * valid, &r.full[st]);
        tc::bulk_load(base + a.stat_off + kStatPitch<kPts, SHIFT>, s + (size_t)a.B * a.npts, 4 * valid, &r.full[st]);
      }
    }
  } else {
    const int rows = BWD ? 2 * a.C + 2 : a.C;
    auto piece = [&](int row, const uint8_t** src, uint32_t* bytes, uint8_t** dst) {
      const uint8_t* from;
      uint32_t len;
      if (row < 2 * a.C && (BWD || row < a.C)) {
        const bool d = row >= a.C;
        const int c = d ? row - a.C : row;
        const T* p = static_cast<const T*>(d ? a.dout : a.x) + ((size_t)b * a.C + c) * a.npts + p0;
        from = reinterpret_cast<const uint8_t*>(p);
        len = valid * (uint32_t)sizeof(T);
        *dst = base + (d ? a.dout_off : 0) + c * kPitch<T, kPts, SHIFT>;
      } else {
        const int s = row - 2 * a.C;
        from = reinterpret_cast<const uint8_t*>(a.stats_in + ((size_t)s * a.B + b) * a.npts + p0);
        len = valid * 4u;
        *dst = base + a.stat_off + s * kStatPitch<kPts, SHIFT>;
      }
      const uint32_t off = (uint32_t)(reinterpret_cast<uintptr_t>(from) & 15);
      *src = from - off;
      *bytes = (off + len + 15) & ~15u;
    };
    uint32_t total = 0;
    const uint8_t* src;
    uint8_t* dst;
    uint32_t bytes;
    for (int row = lane; row < rows; row += 32) {
      piece(row, &src, &bytes, &dst);
      total += bytes;
    }
    tc::mbar_arrive_expect_tx(&r.full[st], total);
    for (int row = lane; row < rows; row += 32) {
      piece(row, &src, &bytes, &dst);
      tc::bulk_load(dst, src, bytes, &r.full[st]);
    }
  }
}

__device__ __forceinline__ Ring ring_setup(const RingArgs& a, uint8_t* smem, int loaders) {
  Ring r;
  r.stage = smem;
  r.full = reinterpret_cast<uint64_t*>(smem + (size_t)a.stages * a.stage_bytes);
  r.empty = r.full + kMaxStages;
  if (threadIdx.x == 0) {
    for (int i = 0; i < a.stages; ++i) {
      tc::mbar_init(&r.full[i], loaders);
      tc::mbar_init(&r.empty[i], kWarps);
    }
    tc::fence_barrier_init();
  }
  __syncthreads();
  return r;
}

__device__ __forceinline__ uint8_t* align128(uint8_t* p) {
  return reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(p) + 127) & ~uintptr_t(127));
}

// Shared memory behind the ring: barriers, gain and bias of every channel, and per group two
// sums per point of each row of lanes and one row of results.
constexpr size_t ring_tail(int C, int pts, int lpr) {
  return 2 * kMaxStages * 8 + 8 * (size_t)C + (size_t)kGroups * (kWarps * (32 / lpr) + 1) * pts * 8;
}

template <typename T, int VEC, int LPR, bool SHIFT>
__global__ void __launch_bounds__(kThreads, 1) norm_ring_fwd_kernel(const __grid_constant__ CUtensorMap map_x,
                                                                    RingArgs a) {
  constexpr int kPts = LPR * VEC, NP = (VEC + 1) / 2, kRows = kWarps * (32 / LPR);
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align128(smem_raw);
  const Ring ring = ring_setup(a, smem, SHIFT ? 32 : 1);
  float2* par = reinterpret_cast<float2*>(ring.empty + kMaxStages);
  float2* red = par + a.C;
  const T* gain = static_cast<const T*>(a.gain);
  const T* bias = static_cast<const T*>(a.bias);
  for (int c = threadIdx.x; c < a.C; c += kThreads)
    par[c] = make_float2(gain ? to_f32(gain[c]) : 1.0f, bias ? to_f32(bias[c]) : 0.0f);
  __syncthreads();
  const int warp = threadIdx.x >> 5;
  if (warp == 0)
    for (int k = 0; k < a.stages; ++k) load_tile<T, kPts, SHIFT, false>(a, &map_x, nullptr, ring, k);
  const int group = warp / kWarps, t = threadIdx.x - group * kGroup;
  const int lane = threadIdx.x % LPR, w = t / LPR;  // row of lanes
  red += group * (kRows + 1) * kPts;
  float2* fin = red + kRows * kPts;
  const int nch = w < a.C ? (a.C - w + kRows - 1) / kRows : 0;
  const float inv_own = nch > 0 ? 1.0f / (float)nch : 0.0f;
  const float inv_c = 1.0f / (float)a.C;
  const int n_lo = a.C / kRows, extra = a.C % kRows;
  int k = group;
  for (long long tile = blockIdx.x + (long long)group * gridDim.x; tile < a.tiles;
       tile += (long long)kGroups * gridDim.x, k += kGroups) {
    const int st = k % a.stages;
    const int b = (int)(tile / a.tiles_per_plane), p0 = (int)(tile % a.tiles_per_plane) * kPts;
    const int valid = min(kPts, a.npts - p0);
    const uint8_t* rows = ring.stage + (size_t)st * a.stage_bytes;
    const size_t at0 = (size_t)b * a.C * a.npts + p0;
    auto row_of = [&](int c) {
      const uint8_t* p = rows + c * kPitch<T, kPts, SHIFT>;
      if (SHIFT) p += past16(static_cast<const T*>(a.x), at0 + (size_t)c * a.npts);
      return p;
    };
    tc::mbar_wait(&ring.full[st], (k / a.stages) & 1);
    F2 s[NP], q[NP], first[NP];
#pragma unroll
    for (int i = 0; i < NP; ++i) s[i] = q[i] = first[i] = pack(0.0f, 0.0f);
    if (nch > 0) {
      read_row<T, VEC, LPR, SHIFT>(row_of(w), lane, first);
#pragma unroll
      for (int i = 0; i < NP; ++i) first[i] = neg2(first[i]);
    }
#pragma unroll 4
    for (int c = w + kRows; c < a.C; c += kRows) {
      F2 v[NP];
      read_row<T, VEC, LPR, SHIFT>(row_of(c), lane, v);
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        v[i] = add2(v[i], first[i]);
        s[i] = add2(s[i], v[i]);
        q[i] = fma2(v[i], v[i], q[i]);
      }
    }
    // point e of a lane sits at e * LPR + lane: free of bank conflicts both ways
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      const F2 mean = fma2(s[i], pack(inv_own, inv_own), neg2(first[i]));   // of the row's channels
      const F2 m2 = fma2(mul2(s[i], pack(-inv_own, -inv_own)), s[i], q[i]);
      const float2 mv = unpack(mean), qv = unpack(m2);
      red[w * kPts + 2 * i * LPR + lane] = make_float2(mv.x, fmaxf(qv.x, 0.0f));
      if (2 * i + 1 < VEC) red[w * kPts + (2 * i + 1) * LPR + lane] = make_float2(mv.y, fmaxf(qv.y, 0.0f));
    }
    tc::named_bar_sync(1 + group, kGroup);
    for (int p = t; p < kPts; p += kGroup) {
      float S = 0.0f;
#pragma unroll
      for (int r = 0; r < kRows; ++r) S = fmaf(red[r * kPts + p].x, (float)(n_lo + (r < extra)), S);
      const float mean = S * inv_c;
      float M = 0.0f;
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        const float2 e = red[r * kPts + p];
        const float d = e.x - mean;
        M += fmaf(d * d, (float)(n_lo + (r < extra)), e.y);
      }
      fin[p] = make_float2(mean, 1.0f / sqrtf(fmaf(M, inv_c, a.eps)));
    }
    tc::named_bar_sync(1 + group, kGroup);
    F2 mr[NP], rr[NP];
    {
      float mean[2 * NP], r[2 * NP];
#pragma unroll
      for (int e = 0; e < 2 * NP; ++e) {
        const float2 f = e < VEC ? fin[e * LPR + lane] : make_float2(0.0f, 0.0f);
        mean[e] = f.x;
        r[e] = f.y;
      }
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        rr[i] = pack(r[2 * i], r[2 * i + 1]);
        mr[i] = pack(-mean[2 * i], -mean[2 * i + 1]);
      }
      if (a.stats && w < 2) {
        float* dst = a.stats + ((size_t)w * a.B + b) * a.npts + p0;
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          const int p = SHIFT ? lane + LPR * e : lane * VEC + e;
          if (p < valid) dst[p] = w == 0 ? mean[e] : r[e];
        }
      }
    }
#pragma unroll 4
    for (int c = w; c < a.C; c += kRows) {
      F2 v[NP];
      read_row<T, VEC, LPR, SHIFT>(row_of(c), lane, v);
      const float2 g = par[c];
      const F2 ga = pack(g.x, g.x), bi = pack(g.y, g.y);
#pragma unroll
      for (int i = 0; i < NP; ++i) v[i] = fma2(mul2(add2(v[i], mr[i]), rr[i]), ga, bi);
      write_row<T, VEC, LPR, SHIFT>(static_cast<T*>(a.out) + at0 + (size_t)c * a.npts, lane, valid, v);
    }
    __syncwarp();
    if ((threadIdx.x & 31) == 0) tc::mbar_arrive(&ring.empty[st]);
    if (t < 32 && tc::mbar_wait(&ring.empty[st], (k / a.stages) & 1))
      load_tile<T, kPts, SHIFT, false>(a, &map_x, nullptr, ring, k + a.stages);
  }
}

// NC: channels per row of lanes, at most.
template <typename T, int VEC, int LPR, int NC, bool SHIFT>
__global__ void __launch_bounds__(kThreads, 1) norm_ring_bwd_kernel(const __grid_constant__ CUtensorMap map_x,
                                                                    const __grid_constant__ CUtensorMap map_d,
                                                                    RingArgs a) {
  constexpr int kPts = LPR * VEC, NP = (VEC + 1) / 2, kRows = kWarps * (32 / LPR);
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align128(smem_raw);
  const Ring ring = ring_setup(a, smem, SHIFT ? 32 : 1);
  float* par = reinterpret_cast<float*>(ring.empty + kMaxStages);
  float2* red = reinterpret_cast<float2*>(par + 2 * a.C);
  const T* gain = static_cast<const T*>(a.gain);
  for (int c = threadIdx.x; c < a.C; c += kThreads) par[c] = gain ? to_f32(gain[c]) : 1.0f;
  __syncthreads();
  const int warp = threadIdx.x >> 5;
  if (warp == 0)
    for (int k = 0; k < a.stages; ++k) load_tile<T, kPts, SHIFT, true>(a, &map_x, &map_d, ring, k);
  const int group = warp / kWarps, t = threadIdx.x - group * kGroup;
  const int lane = threadIdx.x % LPR, w = t / LPR;  // row of lanes
  red += group * (kRows + 1) * kPts;
  float2* fin = red + kRows * kPts;
  const float inv_c = 1.0f / (float)a.C;
  float ag[NC], ab[NC];
#pragma unroll
  for (int i = 0; i < NC; ++i) ag[i] = ab[i] = 0.0f;
  int k = group;
  for (long long tile = blockIdx.x + (long long)group * gridDim.x; tile < a.tiles; tile += (long long)kGroups * gridDim.x, k += kGroups) {
    const int st = k % a.stages;
    const int b = (int)(tile / a.tiles_per_plane), p0 = (int)(tile % a.tiles_per_plane) * kPts;
    const int valid = min(kPts, a.npts - p0);
    const uint8_t* rows = ring.stage + (size_t)st * a.stage_bytes;
    const size_t at0 = (size_t)b * a.C * a.npts + p0;
    tc::mbar_wait(&ring.full[st], (k / a.stages) & 1);
    // xh = x r - mean r; points behind the plane's end have r = mean = 0
    F2 rr[NP], mr[NP], s1[NP], s2[NP];
    {
      float r[2 * NP], m[2 * NP];
#pragma unroll
      for (int e = 0; e < 2 * NP; ++e) {
        r[e] = m[e] = 0.0f;
        const int p = SHIFT ? lane + LPR * e : lane * VEC + e;
        if (e < VEC && p < valid) {
          const uint8_t* sm = rows + a.stat_off;
          const uint8_t* sr = sm + kStatPitch<kPts, SHIFT>;
          if (SHIFT) {
            sm += past16(a.stats_in, (size_t)b * a.npts + p0);
            sr += past16(a.stats_in, ((size_t)a.B + b) * a.npts + p0);
          }
          r[e] = reinterpret_cast<const float*>(sr)[p];
          m[e] = -reinterpret_cast<const float*>(sm)[p] * r[e];
        }
      }
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        rr[i] = pack(r[2 * i], r[2 * i + 1]);
        mr[i] = pack(m[2 * i], m[2 * i + 1]);
        s1[i] = s2[i] = pack(0.0f, 0.0f);
      }
    }
    auto read = [&](int c, F2 (&x)[NP], F2 (&u)[NP]) {
      const uint8_t* px = rows + c * kPitch<T, kPts, SHIFT>;
      const uint8_t* pu = px + a.dout_off;
      if (SHIFT) {
        const size_t at = at0 + (size_t)c * a.npts;
        px += past16(static_cast<const T*>(a.x), at);
        pu += past16(static_cast<const T*>(a.dout), at);
      }
      read_row<T, VEC, LPR, SHIFT>(px, lane, x);
      read_row<T, VEC, LPR, SHIFT>(pu, lane, u);
      if (valid < kPts) {  // whatever lies behind the plane's end counts as zero
#pragma unroll
        for (int i = 0; i < NP; ++i) {
          const int pa = SHIFT ? lane + 2 * LPR * i : lane * VEC + 2 * i, pb = SHIFT ? pa + LPR : pa + 1;
          const float2 fx = unpack(x[i]), fu = unpack(u[i]);
          x[i] = pack(pa < valid ? fx.x : 0.0f, pb < valid ? fx.y : 0.0f);
          u[i] = pack(pa < valid ? fu.x : 0.0f, pb < valid ? fu.y : 0.0f);
        }
      }
    };
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      const int c = w + kRows * j;
      if (c < a.C) {
        F2 x[NP], u[NP];
        read(c, x, u);
        const float g = par[c];
        const F2 ga = pack(g, g);
        F2 tg = pack(ag[j], 0.0f), tb = pack(ab[j], 0.0f);
#pragma unroll
        for (int i = 0; i < NP; ++i) {
          const F2 xh = fma2(x[i], rr[i], mr[i]);
          const F2 e = mul2(u[i], ga);
          tg = fma2(u[i], xh, tg);
          tb = add2(tb, u[i]);
          s1[i] = add2(s1[i], e);
          s2[i] = fma2(e, xh, s2[i]);
        }
        const float2 p = unpack(tg), q = unpack(tb);
        ag[j] = p.x + p.y;
        ab[j] = q.x + q.y;
      }
    }
    if (a.out) {
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        const float2 p = unpack(s1[i]), q = unpack(s2[i]);
        red[w * kPts + 2 * i * LPR + lane] = make_float2(p.x, q.x);
        if (2 * i + 1 < VEC) red[w * kPts + (2 * i + 1) * LPR + lane] = make_float2(p.y, q.y);
      }
      tc::named_bar_sync(1 + group, kGroup);
      for (int p = t; p < kPts; p += kGroup) {
        float x = 0.0f, y = 0.0f;
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
          const float2 e = red[r * kPts + p];
          x += e.x;
          y += e.y;
        }
        fin[p] = make_float2(x * inv_c, y * inv_c);
      }
      tc::named_bar_sync(1 + group, kGroup);
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        const float2 p = fin[2 * i * LPR + lane];
        const float2 q = 2 * i + 1 < VEC ? fin[(2 * i + 1) * LPR + lane] : make_float2(0.0f, 0.0f);
        s1[i] = pack(-p.x, -q.x);
        s2[i] = pack(-p.y, -q.y);
      }
#pragma unroll 4
      for (int c = w; c < a.C; c += kRows) {
        F2 x[NP], u[NP];
        read(c, x, u);
        const float g = par[c];
        const F2 ga = pack(g, g);
#pragma unroll
        for (int i = 0; i < NP; ++i) {
          const F2 xh = fma2(x[i], rr[i], mr[i]);
          x[i] = mul2(rr[i], fma2(xh, s2[i], fma2(u[i], ga, s1[i])));
        }
        write_row<T, VEC, LPR, SHIFT>(static_cast<T*>(a.out) + at0 + (size_t)c * a.npts, lane, valid, x);
      }
    }
    __syncwarp();
    if ((threadIdx.x & 31) == 0) tc::mbar_arrive(&ring.empty[st]);
    if (t < 32 && tc::mbar_wait(&ring.empty[st], (k / a.stages) & 1))
      load_tile<T, kPts, SHIFT, true>(a, &map_x, &map_d, ring, k + a.stages);
  }
  if (!a.part) return;
  // one row of 2C sums per group
  float* row = a.part + ((size_t)blockIdx.x * kGroups + group) * 2 * a.C;
#pragma unroll
  for (int j = 0; j < NC; ++j) {
    const int c = w + kRows * j;
    float g = ag[j], d = ab[j];
#pragma unroll
    for (int m = LPR / 2; m; m >>= 1) {
      g += __shfl_xor_sync(~0u, g, m);
      d += __shfl_xor_sync(~0u, d, m);
    }
    if (lane == 0 && c < a.C) {
      row[c] = g;
      row[a.C + c] = d;
    }
  }
}

// ------------------------------------------------------------------ host side

struct RingPlan {
  bool ok = false;
  int vec = 0, lpr = 0;
  bool shift = false;
  RingArgs a{};
  size_t smem = 0;
  int grid = 0;
};

template <typename T>
RingPlan plan_tile(const NormArgs& n, bool bwd, bool shift, int vec, int lpr, int sms) {
  RingPlan p;
  const int es = (int)sizeof(T), arrays = bwd ? 2 : 1;
  const int pts = vec * lpr;
  const int pitch = pts * es + (shift ? 16 : 0), stat = bwd ? 2 * (pts * 4 + (shift ? 16 : 0)) : 0;
  p.vec = vec;
  p.lpr = lpr;
  p.shift = shift;
  RingArgs& a = p.a;
  a.boxes = n.C > 256 ? 2 : 1;
  if (n.C > 512) return p;
  a.box_rows = (n.C + a.boxes - 1) / a.boxes;
  const int rows = shift ? n.C : a.boxes * a.box_rows;
  auto up128 = [](int v) { return (v + 127) & ~127; };
  a.dout_off = bwd ? up128(rows * pitch) : 0;
  a.stat_off = up128(rows * pitch) * arrays;
  a.stage_bytes = up128(a.stat_off + stat);
  const size_t tail = ring_tail(n.C, pts, lpr) + 128;
  if (tail >= kRingSmem) return p;
  a.stages = (int)std::min<size_t>(kMaxStages, (kRingSmem - tail) / a.stage_bytes);
  a.B = n.B;
  a.C = n.C;
  a.npts = (int)n.npts;
  a.tiles_per_plane = (int)((n.npts + pts - 1) / pts);
  a.tiles = (long long)n.B * a.tiles_per_plane;
  p.smem = (size_t)a.stages * a.stage_bytes + tail;
  p.grid = (int)std::min<long long>(sms, a.tiles);
  // a row of lanes of the backward pass has registers for 16 channels
  p.ok = a.stages >= 3 && (!bwd || n.C <= 16 * kWarps * (32 / lpr));
  return p;
}

template <typename T>
RingPlan plan_ring(const NormArgs& n, bool bwd, int sms) {
  const int es = (int)sizeof(T);
  bool al = n.npts * es % 16 == 0;
  for (const void* q : {n.x, (const void*)n.out, n.dout, (const void*)n.dx, (const void*)n.stats})
    al = al && reinterpret_cast<uintptr_t>(q) % 16 == 0;
  // the widest rows that leave three stages and every SM a tile
  const int shapes[3][2] = {{16 / es, 32}, {16 / es, 16}, {8 / es, 16}};
  RingPlan p;
  for (const auto& v : shapes) {
    RingPlan q = plan_tile<T>(n, bwd, !al, v[0], v[1], sms);
    if (q.ok) p = q;
    if (q.ok && q.a.tiles >= 2 * sms) break;
  }
  return p;
}

bool field_map(CUtensorMap* m, bool bf16, const void* base, const RingArgs& a, int pts) {
  tc::EncodeTiledFn f = tc::encode_tiled_fn();
  if (!f) return false;
  const int es = bf16 ? 2 : 4;
  const cuuint64_t dims[3] = {(cuuint64_t)a.npts, (cuuint64_t)a.C, (cuuint64_t)a.B};
  const cuuint64_t strides[2] = {(cuuint64_t)a.npts * es, (cuuint64_t)a.npts * es * a.C};
  const cuuint32_t box[3] = {(cuuint32_t)pts, (cuuint32_t)a.box_rows, 1}, one[3] = {1, 1, 1};
  return f(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, const_cast<void*>(base),
           dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
           CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename K>
cudaError_t allow_smem(K k, size_t bytes) {
  return cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
}

template <typename T, int VEC, int LPR, bool SHIFT>
cudaError_t run_fwd(const RingPlan& p, const CUtensorMap& mx, cudaStream_t st) {
  auto k = norm_ring_fwd_kernel<T, VEC, LPR, SHIFT>;
  cudaError_t e = allow_smem(k, p.smem);
  if (e != cudaSuccess) return e;
  k<<<p.grid, kThreads, p.smem, st>>>(mx, p.a);
  count_launch();
  return cudaGetLastError();
}

template <typename T, int VEC, int LPR, int NC, bool SHIFT>
cudaError_t run_bwd(const RingPlan& p, const CUtensorMap& mx, const CUtensorMap& md, cudaStream_t st) {
  auto k = norm_ring_bwd_kernel<T, VEC, LPR, NC, SHIFT>;
  cudaError_t e = allow_smem(k, p.smem);
  if (e != cudaSuccess) return e;
  k<<<p.grid, kThreads, p.smem, st>>>(mx, md, p.a);
  count_launch();
  return cudaGetLastError();
}

template <typename T, int VEC, int LPR, bool SHIFT>
cudaError_t run_shape(const RingPlan& p, bool bwd, const CUtensorMap& mx, const CUtensorMap& md, cudaStream_t st) {
  if (!bwd) return run_fwd<T, VEC, LPR, SHIFT>(p, mx, st);
  const int rows = kWarps * (32 / LPR), nc = (p.a.C + rows - 1) / rows;
  if (nc <= 4) return run_bwd<T, VEC, LPR, 4, SHIFT>(p, mx, md, st);
  if (nc <= 8) return run_bwd<T, VEC, LPR, 8, SHIFT>(p, mx, md, st);
  return run_bwd<T, VEC, LPR, 16, SHIFT>(p, mx, md, st);
}

template <typename T, bool SHIFT>
cudaError_t run_plan(const RingPlan& p, bool bwd, const CUtensorMap& mx, const CUtensorMap& md, cudaStream_t st) {
  constexpr int es = (int)sizeof(T);
  if (p.lpr == 32) return run_shape<T, 16 / es, 32, SHIFT>(p, bwd, mx, md, st);
  if (p.vec * es == 16) return run_shape<T, 16 / es, 16, SHIFT>(p, bwd, mx, md, st);
  return run_shape<T, 8 / es, 16, SHIFT>(p, bwd, mx, md, st);
}

template <typename T>
bool ring_run(const NormArgs& n, bool bwd, int sms, cudaStream_t st, int* rows, cudaError_t* err) {
  if (n.npts < 64 || (bwd && n.C > 16 * kWarps * 2)) return false;
  RingPlan p = plan_ring<T>(n, bwd, sms);
  if (!p.ok) return false;
  RingArgs& a = p.a;
  a.x = n.x;
  a.dout = n.dout;
  a.gain = n.gain;
  a.bias = n.bias;
  a.eps = n.eps;
  a.out = bwd ? n.dx : n.out;
  a.stats = n.stats;
  a.stats_in = n.stats;
  a.part = n.dgain || n.dbias ? n.part : nullptr;
  CUtensorMap mx{}, md{};
  const bool bf16 = sizeof(T) == 2;
  if (!p.shift && (!field_map(&mx, bf16, n.x, a, p.lpr * p.vec) || (bwd && !field_map(&md, bf16, n.dout, a, p.lpr * p.vec)))) {
    *err = cudaErrorInvalidValue;
    return true;
  }
  *rows = kGroups * p.grid;
  *err = p.shift ? run_plan<T, true>(p, bwd, mx, md, st) : run_plan<T, false>(p, bwd, mx, md, st);
  return true;
}

}  // namespace

bool launch_norm_ring(bool bf16, const NormArgs& a, bool bwd, int sms, cudaStream_t st, int* rows, cudaError_t* err) {
  return bf16 ? ring_run<__nv_bfloat16>(a, bwd, sms, st, rows, err) : ring_run<float>(a, bwd, sms, st, rows, err);
}

int take_norm_status() {
  int v = 0, z = 0;
  cudaMemcpyFromSymbol(&v, g_device_status, sizeof(int));
  if (v) cudaMemcpyToSymbol(g_device_status, &z, sizeof(int));
  return v;
}

}  // namespace disco
