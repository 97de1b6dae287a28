// Layer norm over channels for long planes: the tiles of x (and dout) pass through a ring in
// shared memory.  Formulas and sums as in norm.cu.
//
// What bounds both passes is HBM, and what kept the register form below it was latency: its
// loads are only in flight between two barriers of a CTA.  Here a ring of tiles of C channels x
// LPR * VEC points is kept full while G groups of W = 1 to 16 warps take the tiles in turn.  A tile
// is read from HBM once and from shared memory once: its sums are added on the way into registers
// (at most 32 of packed values a thread), the stage is free for the next tile at once, and the
// result is formed from the registers after the sums over channels have crossed the group.
// The number of stages is a multiple of the number of groups, so each stage has one group's tiles.
// LPR = 32, 16 or 8 lanes take a channel row, VEC points each, so a group has W * 32 / LPR rows of
// lanes and row r takes the channels r, r + rows, ....  Few channels take small groups (one warp
// has no barrier at all), many take large ones.
//
// Loads.  GRAN = 16 (every plane starts on 16 bytes): one TMA box of C rows per array, issued by
// the first warp of the group that has read the stage.  GRAN = 4 or 2 (planes start on any
// 4 or 2 bytes): every row of lanes copies its own channels' rows of its group's next tile with
// cp.async, as the 16-byte blocks that hold a value of the row's piece (so a copy may take in up to
// 15 bytes before and behind it, never a block without a value), and reads them from their own
// offset, GRAN bytes at a time.  No other warp reads these rows, so they need no barrier.
//
// Forward sums in one pass: a row of lanes adds v = x - k and v^2 about the value k of its first
// channel.  k is one of the n values it adds, so (mean - k)^2 is at most n times their variance and
// m2 = sum v^2 - (sum v)^2 / n loses at most log2(n) + 1 bits; the rows then combine as in norm.cu.
//
// xh is (x - mean) r, not x r - mean r: a difference near the mean is exact, while rounding mean r is
// off by u |mean| r, which for points of equal channels (r = 1 / sqrt(eps)) gave 0.1 instead of 0.  The
// third instruction an element takes the backward pass of 64 bf16 channels at 721 x 1440 from 91 to 93 us.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "common.cuh"
#include "kernels.h"
#include "norm.h"
#include "norm_partial.cuh"
#include "tc_common.cuh"

namespace disco {
namespace {

constexpr int kThreads = 512;  // 128 registers a thread
constexpr int kMaxStages = 32;
constexpr size_t kRingSmem = 225 * 1024;  // of 227 KB

// Two fp32 values of neighbouring points.
struct F2 {
  float x, y;
};
__device__ __forceinline__ F2 twice(float a) { return F2{a, a}; }
__device__ __forceinline__ F2 add2(F2 a, F2 b) { return F2{a.x + b.x, a.y + b.y}; }
__device__ __forceinline__ F2 mul2(F2 a, F2 b) { return F2{a.x * b.x, a.y * b.y}; }
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) { return F2{fmaf(a.x, b.x, c.x), fmaf(a.y, b.y, c.y)}; }
__device__ __forceinline__ F2 neg2(F2 a) { return F2{-a.x, -a.y}; }

struct RingArgs {
  int B, C;
  int npts;
  int tiles_per_plane;
  long long tiles;
  int stages, stage_bytes;
  int dout_off, stat_off;      // byte offsets in a stage: dout rows, statistics rows (GRAN 16)
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

// The form of a kernel: its lanes and groups, and which points of the tile a lane's values are.
// FULL: every row of lanes has exactly NC channels, so no channel needs a guard.
template <typename T_, int VEC_, int LPR_, int W_, int NC_, int GRAN_, bool FULL_ = false>
struct Form {
  using T = T_;
  static constexpr int VEC = VEC_, LPR = LPR_, W = W_, GRAN = GRAN_;
  static constexpr int NC = NC_;  // channels per row of lanes, at most
  static constexpr int kGroup = W * 32, G = kThreads / kGroup;
  static constexpr int kPts = LPR * VEC, NP = VEC / 2;
  static constexpr int kRows = W * (32 / LPR);
  static constexpr bool kTma = GRAN == 16, kFull = FULL_;
  using Filled = Form<T_, VEC_, LPR_, W_, NC_, GRAN_, true>;
  static constexpr int kWords = VEC * (int)sizeof(T) / 4;  // packed values of a lane and channel
  // consecutive points a lane reads at once
  static constexpr int kRun = kTma ? VEC : (GRAN < (int)sizeof(T) ? 1 : GRAN / (int)sizeof(T));
  static constexpr int kPitch = kPts * (int)sizeof(T) + (kTma ? 0 : 16);
  // the sums of a point are joined by kJoin lanes; rows of sums are kSumPitch apart, which keeps
  // those lanes on different banks
  static constexpr int kJoin = kGroup > kPts ? kGroup / kPts : 1, kSumPitch = kPts + (kJoin < 16 ? 16 / kJoin : 1);
  static_assert(VEC % 2 == 0 && VEC % kRun == 0 && kJoin <= 32 && kRows % kJoin == 0 && kPts % (kGroup / kJoin) == 0, "shape");
  // the tile's point that value e of a lane is
  static __device__ __forceinline__ int point(int lane, int e) {
    return (lane + LPR * (e / kRun)) * kRun + e % kRun;
  }
};

template <typename F>
__device__ __forceinline__ void read_row(const uint8_t* row, int lane, uint32_t (&v)[F::kWords]) {
  using T = typename F::T;
  constexpr int kBytes = F::kRun * (int)sizeof(T);
#pragma unroll
  for (int g = 0; g < F::VEC / F::kRun; ++g) {
    const uint8_t* p = row + (lane + F::LPR * g) * kBytes;
    if constexpr (kBytes == 2) {
      const uint32_t h = *reinterpret_cast<const uint16_t*>(p);
      if (g % 2 == 0) v[g / 2] = h;
      else v[g / 2] |= h << 16;
    } else if constexpr (kBytes == 4) {
      v[g] = *reinterpret_cast<const uint32_t*>(p);
    } else if constexpr (kBytes == 8) {
      const uint2 q = *reinterpret_cast<const uint2*>(p);
      v[0] = q.x;
      v[1] = q.y;
    } else {
      const uint4 q = *reinterpret_cast<const uint4*>(p);
      v[0] = q.x;
      v[1] = q.y;
      v[2] = q.z;
      v[3] = q.w;
    }
  }
}

// Pair k of a lane's values.
template <typename F>
__device__ __forceinline__ F2 pair_of(const uint32_t (&v)[F::kWords], int k) {
  if constexpr (sizeof(typename F::T) == 2) return F2{__uint_as_float(v[k] << 16), __uint_as_float(v[k] & 0xffff0000u)};
  else return F2{__uint_as_float(v[2 * k]), __uint_as_float(v[2 * k + 1])};
}

template <typename F>
__device__ __forceinline__ void write_row(typename F::T* dst, int lane, int valid, const F2 (&v)[F::NP]) {
  using T = typename F::T;
  constexpr int kBytes = F::kRun * (int)sizeof(T);
  uint32_t w[F::kWords];
#pragma unroll
  for (int k = 0; k < F::NP; ++k) {
    const F2 q = v[k];
    if constexpr (sizeof(T) == 2) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(q.x, q.y);
      w[k] = *reinterpret_cast<const uint32_t*>(&h);
    } else {
      w[2 * k] = __float_as_uint(q.x);
      w[2 * k + 1] = __float_as_uint(q.y);
    }
  }
#pragma unroll
  for (int g = 0; g < F::VEC / F::kRun; ++g) {
    const int p = (lane + F::LPR * g) * F::kRun;
    if (p >= valid) continue;  // planes are whole runs long
    if constexpr (kBytes == 2) *reinterpret_cast<uint16_t*>(dst + p) = (uint16_t)(w[g / 2] >> (16 * (g % 2)));
    else if constexpr (kBytes == 4) *reinterpret_cast<uint32_t*>(dst + p) = w[g];
    else if constexpr (kBytes == 8) *reinterpret_cast<uint2*>(dst + p) = make_uint2(w[0], w[1]);
    else *reinterpret_cast<uint4*>(dst + p) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

struct Ring {
  uint8_t* stage;
  uint64_t* full;
  uint64_t* empty;
};

struct Tile {
  int b, p0, valid;
  size_t at;  // of channel 0
};

template <typename F>
__device__ __forceinline__ Tile tile_of(const RingArgs& a, long long tile) {
  Tile t;
  t.b = (int)(tile / a.tiles_per_plane);
  t.p0 = (int)(tile % a.tiles_per_plane) * F::kPts;
  t.valid = min(F::kPts, a.npts - t.p0);
  t.at = (size_t)t.b * a.C * a.npts + t.p0;
  return t;
}

// GRAN 16, one warp: tile k of this CTA into stage k % stages, which is free.
template <typename F, bool BWD>
__device__ __forceinline__ void load_boxes(const RingArgs& a, const CUtensorMap* map_x, const CUtensorMap* map_d,
                                           const Ring& r, int k) {
  const long long tile = blockIdx.x + (long long)k * gridDim.x;
  if (tile >= a.tiles || (threadIdx.x & 31) != 0) return;
  const int st = k % a.stages;
  const Tile t = tile_of<F>(a, tile);
  uint8_t* base = r.stage + (size_t)st * a.stage_bytes;
  const uint32_t rows = (uint32_t)(a.boxes * a.box_rows * F::kPitch);
  tc::mbar_arrive_expect_tx(&r.full[st], BWD ? 2 * rows + 8u * t.valid : rows);
  for (int i = 0; i < a.boxes; ++i) {
    tc::tma_load_3d(base + i * a.box_rows * F::kPitch, map_x, &r.full[st], t.p0, i * a.box_rows, t.b);
    if (BWD)
      tc::tma_load_3d(base + a.dout_off + i * a.box_rows * F::kPitch, map_d, &r.full[st], t.p0, i * a.box_rows, t.b);
  }
  if (BWD) {
    const float* s = a.stats_in + (size_t)t.b * a.npts + t.p0;
    tc::bulk_load(base + a.stat_off, s, 4 * t.valid, &r.full[st]);
    tc::bulk_load(base + a.stat_off + 4 * F::kPts, s + (size_t)a.B * a.npts, 4 * t.valid, &r.full[st]);
  }
}

// GRAN < 16: this row of lanes' channels of tile k, one group of asynchronous copies per call.
template <typename F, bool BWD>
__device__ __forceinline__ void load_rows(const RingArgs& a, const Ring& r, int k, int lane, int w) {
  using T = typename F::T;
  const long long tile = blockIdx.x + (long long)k * gridDim.x;
  if (tile < a.tiles) {
    const Tile t = tile_of<F>(a, tile);
    uint8_t* base = r.stage + (size_t)(k % a.stages) * a.stage_bytes;
    // the 32 / LPR rows of lanes of a warp have neighbouring channels; all its lanes copy together
    constexpr int kBlocks = F::kPitch / 16, kSide = 32 / F::LPR;
    const int wlane = threadIdx.x & 31;
    for (int c0 = w - (wlane / F::LPR); c0 < a.C; c0 += F::kRows) {
#pragma unroll
      for (int i = wlane; i < kBlocks * kSide; i += 32) {
        const int c = c0 + i / kBlocks, blk = i % kBlocks;
        if (c >= a.C) break;
#pragma unroll
        for (int arr = 0; arr < (BWD ? 2 : 1); ++arr) {
          const uint8_t* p =
              reinterpret_cast<const uint8_t*>(static_cast<const T*>(arr ? a.dout : a.x) + t.at + (size_t)c * a.npts);
          const uint32_t off = (uint32_t)(reinterpret_cast<uintptr_t>(p) & 15);
          if (16 * blk < (int)(off + t.valid * (uint32_t)sizeof(T)))
            tc::cp_async16(base + (arr ? a.dout_off : 0) + c * F::kPitch + 16 * blk, p - off + 16 * blk, 16);
        }
      }
    }
  }
  tc::cp_async_commit();
}

// Waits until at most `most` of this thread's groups of copies are in flight.
__device__ __forceinline__ void wait_rows(int most) {
  if (most <= 0) tc::cp_async_wait<0>();
  else if (most == 1) tc::cp_async_wait<1>();
  else if (most == 2) tc::cp_async_wait<2>();
  else tc::cp_async_wait<3>();
  __syncwarp();
}

template <typename F>
__device__ __forceinline__ Ring ring_setup(const RingArgs& a, uint8_t* smem) {
  Ring r;
  r.stage = smem;
  r.full = reinterpret_cast<uint64_t*>(smem + (size_t)a.stages * a.stage_bytes);
  r.empty = r.full + kMaxStages;
  if (F::kTma && threadIdx.x == 0) {
    for (int i = 0; i < a.stages; ++i) {
      tc::mbar_init(&r.full[i], 1);
      tc::mbar_init(&r.empty[i], F::W);
    }
    tc::fence_barrier_init();
  }
  return r;
}

__device__ __forceinline__ uint8_t* align128(uint8_t* p) {
  return reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(p) + 127) & ~uintptr_t(127));
}

// Shared memory behind the ring: barriers, gain and bias of every channel (backward: gain, and per group
// 2C fp64 sums over points), and per group two sums per point of each row of lanes and one row of results.
template <typename F, bool BWD>
constexpr size_t ring_tail(int C) {
  return 2 * kMaxStages * 8 + (8 + (BWD ? 16 * F::G : 0)) * (size_t)C + (size_t)F::G * (F::kRows * F::kSumPitch + F::kPts) * 8;
}

// Tiles whose parameter sums a thread adds in fp32 before they go on in fp64.  Going on with every tile
// took the bf16 backward of 64 channels at 721 x 1440 from 93 to 109 us (conversions), this none; that of
// 256 channels, one group of warps at a time, 2 x 361 x 720, goes from 173 to 181.
constexpr int kFlush = 8;

// Bytes by which element `at` of an array at `base` lies past a 16-byte boundary (0 for GRAN 16).
template <typename F>
__device__ __forceinline__ uint32_t past16(const void* base, size_t at) {
  if (F::kTma) return 0;
  return ((uint32_t)reinterpret_cast<uintptr_t>(base) + (uint32_t)at * (uint32_t)sizeof(typename F::T)) & 15u;
}

// What a group does when it has read stage st: the next tile comes into its place.  A box is written
// by the async proxy, which an arrival alone does not order behind this proxy's reads: without the
// fence the last loads of a busy SM were still in flight when the next tile landed (64 bytes of a
// channel from tile k + stages, in 1 of some 300 calls of one form).  Rows copied by cp.async need none:
// the copies are this proxy's, and a warp's own.
template <typename F, bool BWD>
__device__ __forceinline__ void release(const RingArgs& a, const CUtensorMap* map_x, const CUtensorMap* map_d,
                                        const Ring& r, int k, int st, int t, int lane, int w, bool ok) {
  if (F::kTma) tc::fence_proxy_async();
  __syncwarp();
  if (F::kTma) {
    if ((threadIdx.x & 31) == 0) tc::mbar_arrive(&r.empty[st]);
    if (t < 32 && ok && tc::mbar_wait(&r.empty[st], (k / a.stages) & 1)) load_boxes<F, BWD>(a, map_x, map_d, r, k + a.stages);
  } else {
    load_rows<F, BWD>(a, r, k + a.stages, lane, w);
  }
}

template <typename F, bool BWD>
__device__ __forceinline__ void fill_ring(const RingArgs& a, const CUtensorMap* map_x, const CUtensorMap* map_d,
                                          const Ring& r, int group, int lane, int w) {
  if (F::kTma) {
    if (threadIdx.x < 32)
      for (int k = 0; k < a.stages; ++k) load_boxes<F, BWD>(a, map_x, map_d, r, k);
  } else {
    for (int k = group; k < a.stages; k += F::G) load_rows<F, BWD>(a, r, k, lane, w);
  }
}

template <typename F>
__device__ __forceinline__ void group_sync(int group) {
  if constexpr (F::W == 1) __syncwarp();
  else tc::named_bar_sync(1 + group, F::kGroup);
}

template <typename F>
__device__ __forceinline__ float join(float v) {
#pragma unroll
  for (int m = 1; m < F::kJoin; m <<= 1) v += __shfl_xor_sync(~0u, v, m);
  return v;
}

template <typename F>
__global__ void __launch_bounds__(kThreads, 1)
    norm_ring_fwd_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ RingArgs a) {
  using T = typename F::T;
  constexpr int NP = F::NP, VEC = F::VEC, LPR = F::LPR, kPts = F::kPts, kRows = F::kRows, G = F::G, NC = F::NC;
  extern __shared__ uint8_t smem_raw[];
  const Ring ring = ring_setup<F>(a, align128(smem_raw));
  float2* par = reinterpret_cast<float2*>(ring.empty + kMaxStages);
  const T* gain = static_cast<const T*>(a.gain);
  const T* bias = static_cast<const T*>(a.bias);
  for (int c = threadIdx.x; c < a.C; c += kThreads)
    par[c] = make_float2(gain ? to_f32(gain[c]) : 1.0f, bias ? to_f32(bias[c]) : 0.0f);
  __syncthreads();
  const int group = threadIdx.x / F::kGroup, t = threadIdx.x % F::kGroup;
  const int lane = threadIdx.x % LPR, w = t / LPR;  // row of lanes
  fill_ring<F, false>(a, &map_x, nullptr, ring, group, lane, w);
  float2* red = reinterpret_cast<float2*>(par + a.C) + group * (kRows * F::kSumPitch + kPts);
  float2* fin = red + kRows * F::kSumPitch;
  const int nch = w < a.C ? (a.C - w + kRows - 1) / kRows : 0;
  const float inv_own = nch > 0 ? 1.0f / (float)nch : 0.0f;
  const float inv_c = 1.0f / (float)a.C;
  const int n_lo = a.C / kRows, extra = a.C % kRows;
  int k = group;
  bool ok = true;
  for (long long tile = blockIdx.x + (long long)group * gridDim.x; tile < a.tiles;
       tile += (long long)G * gridDim.x, k += G) {
    const int st = k % a.stages;
    const Tile tl = tile_of<F>(a, tile);
    const uint8_t* rows = ring.stage + (size_t)st * a.stage_bytes;
    if (F::kTma) ok = ok && tc::mbar_wait(&ring.full[st], (k / a.stages) & 1);
    else wait_rows(a.stages / G - 1);
    uint32_t raw[NC][F::kWords];
    F2 s[NP], q[NP], first[NP];
#pragma unroll
    for (int i = 0; i < NP; ++i) s[i] = q[i] = first[i] = F2{0.0f, 0.0f};
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      const int c = w + kRows * j;
      if (F::kFull || c < a.C) read_row<F>(rows + c * F::kPitch + past16<F>(a.x, tl.at + (size_t)c * a.npts), lane, raw[j]);
    }
    release<F, false>(a, &map_x, nullptr, ring, k, st, t, lane, w, ok);
    if (F::kFull || nch > 0) {
#pragma unroll
      for (int i = 0; i < NP; ++i) first[i] = neg2(pair_of<F>(raw[0], i));
    }
#pragma unroll
    for (int j = 1; j < NC; ++j) {
      if (F::kFull || j < nch) {
#pragma unroll
        for (int i = 0; i < NP; ++i) {
          const F2 v = add2(pair_of<F>(raw[j], i), first[i]);
          s[i] = add2(s[i], v);
          q[i] = fma2(v, v, q[i]);
        }
      }
    }
    // value e of a lane sits at e * LPR + lane
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      const F2 mean = fma2(s[i], twice(inv_own), neg2(first[i]));  // of the row's channels
      const F2 m2 = fma2(mul2(s[i], twice(-inv_own)), s[i], q[i]);
      const F2 mv = mean, qv = m2;
      red[w * F::kSumPitch + 2 * i * LPR + lane] = make_float2(mv.x, qv.x);
      red[w * F::kSumPitch + (2 * i + 1) * LPR + lane] = make_float2(mv.y, qv.y);
    }
    group_sync<F>(group);
#pragma unroll
    for (int p = t / F::kJoin; p < kPts; p += F::kGroup / F::kJoin) {
      const int sub = t % F::kJoin;
      float2 e[kRows / F::kJoin];
      float S = 0.0f, M = 0.0f;
      const float of = red[p].x;  // row 0 has channels: equal means of rows add up to nothing
#pragma unroll
      for (int r = 0; r < kRows / F::kJoin; ++r) {
        const int row = sub + F::kJoin * r;
        e[r] = red[row * F::kSumPitch + p];
        S = fmaf(e[r].x - of, (float)(n_lo + (row < extra)), S);
      }
      const float mean = fmaf(join<F>(S), inv_c, of);
#pragma unroll
      for (int r = 0; r < kRows / F::kJoin; ++r) {
        const float n = (float)(n_lo + (sub + F::kJoin * r < extra)), d = n > 0.0f ? e[r].x - mean : 0.0f;
        // rounding may leave m2 of equal values a little below zero
        M += fmaf(d * d, n, e[r].y < 0.0f ? 0.0f : e[r].y);
      }
      M = join<F>(M);
      if (sub == 0) fin[p] = make_float2(mean, 1.0f / sqrtf(fmaf(M, inv_c, a.eps)));
    }
    group_sync<F>(group);
    F2 nm[NP], rr[NP];  // -mean, r
    {
      float mean[VEC], r[VEC];
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const float2 f = fin[e * LPR + lane];
        mean[e] = f.x;
        r[e] = f.y;
      }
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        rr[i] = F2{r[2 * i], r[2 * i + 1]};
        nm[i] = F2{-mean[2 * i], -mean[2 * i + 1]};
      }
      for (int which = w; a.stats && which < 2; which += kRows) {
        float* dst = a.stats + ((size_t)which * a.B + tl.b) * a.npts + tl.p0;
        float v[VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e) v[e] = which == 0 ? mean[e] : r[e];
        if constexpr (F::kTma) {  // planes are whole vectors long
          if (lane * VEC < tl.valid) {
#pragma unroll
            for (int e = 0; e < VEC; e += (VEC < 4 ? 2 : 4)) {
              if constexpr (VEC < 4) *reinterpret_cast<float2*>(dst + lane * VEC + e) = make_float2(v[e], v[e + 1]);
              else *reinterpret_cast<float4*>(dst + lane * VEC + e) = make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
            }
          }
        } else {
#pragma unroll
          for (int e = 0; e < VEC; ++e)
            if (F::point(lane, e) < tl.valid) dst[F::point(lane, e)] = v[e];
        }
      }
    }
    T* out = static_cast<T*>(a.out) + tl.at;
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      const int c = w + kRows * j;
      if (F::kFull || c < a.C) {
        const float2 g = par[c];
        const F2 ga = twice(g.x), bi = twice(g.y);
        F2 v[NP];
#pragma unroll
        for (int i = 0; i < NP; ++i) v[i] = fma2(mul2(add2(pair_of<F>(raw[j], i), nm[i]), rr[i]), ga, bi);
        write_row<F>(out + (size_t)c * a.npts, lane, tl.valid, v);
      }
    }
  }
  // after a wait that ran out (the status word says so, the results are void) a warp waits and loads no
  // more, which ends the kernel soon
  if (F::kTma && !ok) tc::give_up();
}

template <typename F>
__global__ void __launch_bounds__(kThreads, 1)
    norm_ring_bwd_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_d,
                         const __grid_constant__ RingArgs a) {
  using T = typename F::T;
  constexpr int NP = F::NP, VEC = F::VEC, LPR = F::LPR, kPts = F::kPts, kRows = F::kRows, G = F::G, NC = F::NC;
  extern __shared__ uint8_t smem_raw[];
  const Ring ring = ring_setup<F>(a, align128(smem_raw));
  float* par = reinterpret_cast<float*>(ring.empty + kMaxStages);
  const T* gain = static_cast<const T*>(a.gain);
  double* sums = reinterpret_cast<double*>(par + 2 * a.C);  // over points: [group][2C]
  for (int c = threadIdx.x; c < a.C; c += kThreads) par[c] = gain ? to_f32(gain[c]) : 1.0f;
  for (int i = threadIdx.x; i < G * 2 * a.C; i += kThreads) sums[i] = 0.0;
  __syncthreads();
  const int group = threadIdx.x / F::kGroup, t = threadIdx.x % F::kGroup;
  const int lane = threadIdx.x % LPR, w = t / LPR;  // row of lanes
  fill_ring<F, true>(a, &map_x, &map_d, ring, group, lane, w);
  float2* red = reinterpret_cast<float2*>(sums + G * 2 * a.C) + group * (kRows * F::kSumPitch + kPts);
  float2* fin = red + kRows * F::kSumPitch;
  const float inv_c = 1.0f / (float)a.C;
  float ag[NC], ab[NC];  // sums over points of `held` tiles
#pragma unroll
  for (int i = 0; i < NC; ++i) ag[i] = ab[i] = 0.0f;
  int held = 0;
  // The 2 NC sums of a row of lanes are added and spread over its lanes in one go (a lane keeps half of
  // the values at each step), and each lane adds its own to the group's: no other row has its channels.
  auto flush = [&]() {
    float v[2 * NC];
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      v[j] = ag[j];
      v[NC + j] = ab[j];
      ag[j] = ab[j] = 0.0f;
    }
    int left = 2 * NC, at = 0;
    bool mine = true;
#pragma unroll
    for (int m = LPR / 2; m; m >>= 1) {
      const bool up = lane & m;
      if (left > 1) {
        left /= 2;
        at += up ? left : 0;
#pragma unroll
        for (int i = 0; i < NC; ++i)
          if (i < left) {
            const float keep = up ? v[left + i] : v[i], give = up ? v[i] : v[left + i];
            v[i] = keep + __shfl_xor_sync(~0u, give, m);
          }
      } else {
        v[0] += __shfl_xor_sync(~0u, v[0], m);
        mine = mine && !up;
      }
    }
#pragma unroll
    for (int i = 0; i < NC; ++i)
      if (i < left && mine) {
        const int c = w + kRows * ((at + i) % NC);
        if (c < a.C) sums[(group * 2 + (at + i) / NC) * a.C + c] += (double)v[i];
      }
    held = 0;
  };
  // GRAN < 16: the statistics of a tile are fetched while the tile before it is finished
  float mean[VEC], rstd[VEC];
  auto fetch_stats = [&](long long tile) {
    const Tile tl = tile_of<F>(a, tile);
    const float* p = a.stats_in + (size_t)tl.b * a.npts + tl.p0;
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      const bool in = tile < a.tiles && F::point(lane, e) < tl.valid;
      mean[e] = in ? p[F::point(lane, e)] : 0.0f;
      rstd[e] = in ? p[(size_t)a.B * a.npts + F::point(lane, e)] : 0.0f;
    }
  };
  int k = group;
  bool ok = true;
  const long long tile0 = blockIdx.x + (long long)group * gridDim.x;
  if (!F::kTma) fetch_stats(tile0);
  for (long long tile = tile0; tile < a.tiles; tile += (long long)G * gridDim.x, k += G) {
    const int st = k % a.stages;
    const Tile tl = tile_of<F>(a, tile);
    const uint8_t* rows = ring.stage + (size_t)st * a.stage_bytes;
    if (F::kTma) {
      ok = ok && tc::mbar_wait(&ring.full[st], (k / a.stages) & 1);
      const float* sm = reinterpret_cast<const float*>(rows + a.stat_off) + lane * VEC;
      const bool in = lane * VEC < tl.valid;  // planes are whole vectors long
#pragma unroll
      for (int e = 0; e < VEC; e += 2) {
        const float2 m = *reinterpret_cast<const float2*>(sm + e);
        const float2 r = *reinterpret_cast<const float2*>(sm + kPts + e);
        mean[e] = in ? m.x : 0.0f;
        mean[e + 1] = in ? m.y : 0.0f;
        rstd[e] = in ? r.x : 0.0f;
        rstd[e + 1] = in ? r.y : 0.0f;
      }
    } else {
      wait_rows(a.stages / G - 1);
    }
    // points behind the plane's end have r = mean = 0
    F2 rr[NP], nm[NP], s1[NP], s2[NP];
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      rr[i] = F2{rstd[2 * i], rstd[2 * i + 1]};
      nm[i] = F2{-mean[2 * i], -mean[2 * i + 1]};
      s1[i] = s2[i] = F2{0.0f, 0.0f};
    }
    uint32_t x[NC][F::kWords], u[NC][F::kWords];
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      const int c = w + kRows * j;
      if (F::kFull || c < a.C) {
        const uint8_t* row = rows + c * F::kPitch;
        const size_t at = tl.at + (size_t)c * a.npts;
        read_row<F>(row + past16<F>(a.x, at), lane, x[j]);
        read_row<F>(row + a.dout_off + past16<F>(a.dout, at), lane, u[j]);
        if (tl.valid < kPts) {  // whatever lies behind the plane's end counts as zero
#pragma unroll
          for (int e = 0; e < VEC; ++e)
            if (F::point(lane, e) >= tl.valid) {
              const uint32_t keep = sizeof(T) == 4 ? 0u : (e % 2 ? 0xffffu : 0xffff0000u);
              constexpr int per = 4 / (int)sizeof(T);
              x[j][e / per] &= keep;
              u[j][e / per] &= keep;
            }
        }
      }
    }
    release<F, true>(a, &map_x, &map_d, ring, k, st, t, lane, w, ok);
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      const int c = w + kRows * j;
      if (F::kFull || c < a.C) {
        const F2 ga = twice(par[c]);
        F2 tg = twice(0.0f), tb = twice(0.0f);
#pragma unroll
        for (int i = 0; i < NP; ++i) {
          const F2 ui = pair_of<F>(u[j], i);
          const F2 xh = mul2(add2(pair_of<F>(x[j], i), nm[i]), rr[i]);
          const F2 e = mul2(ui, ga);
          tg = fma2(ui, xh, tg);
          tb = add2(tb, ui);
          s1[i] = add2(s1[i], e);
          s2[i] = fma2(e, xh, s2[i]);
        }
        const F2 p = tg, q = tb;
        ag[j] += p.x + p.y;
        ab[j] += q.x + q.y;
      }
    }
    if (a.part && ++held == kFlush) flush();
    if (!F::kTma) fetch_stats(tile + (long long)G * gridDim.x);
    if (!a.out) continue;
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      const F2 p = s1[i], q = s2[i];
      red[w * F::kSumPitch + 2 * i * LPR + lane] = make_float2(p.x, q.x);
      red[w * F::kSumPitch + (2 * i + 1) * LPR + lane] = make_float2(p.y, q.y);
    }
    group_sync<F>(group);
#pragma unroll
    for (int p = t / F::kJoin; p < kPts; p += F::kGroup / F::kJoin) {
      const int sub = t % F::kJoin;
      float y = 0.0f, z = 0.0f;
#pragma unroll
      for (int r = 0; r < kRows / F::kJoin; ++r) {
        const float2 e = red[(sub + F::kJoin * r) * F::kSumPitch + p];
        y += e.x;
        z += e.y;
      }
      y = join<F>(y);
      z = join<F>(z);
      if (sub == 0) fin[p] = make_float2(y * inv_c, z * inv_c);
    }
    group_sync<F>(group);
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      const float2 p = fin[2 * i * LPR + lane];
      const float2 q = fin[(2 * i + 1) * LPR + lane];
      s1[i] = F2{-p.x, -q.x};
      s2[i] = F2{-p.y, -q.y};
    }
    T* out = static_cast<T*>(a.out) + tl.at;
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      const int c = w + kRows * j;
      if (F::kFull || c < a.C) {
        const F2 ga = twice(par[c]);
        F2 o[NP];
#pragma unroll
        for (int i = 0; i < NP; ++i) {
          const F2 xh = mul2(add2(pair_of<F>(x[j], i), nm[i]), rr[i]);
          o[i] = mul2(rr[i], fma2(xh, s2[i], fma2(pair_of<F>(u[j], i), ga, s1[i])));
        }
        write_row<F>(out + (size_t)c * a.npts, lane, tl.valid, o);
      }
    }
  }
  // after a wait that ran out (the status word says so, the results are void) a warp waits and loads no
  // more, which ends the kernel soon
  if (F::kTma && !ok) tc::give_up();
  if (!a.part) return;
  flush();
  __syncthreads();
  // one row of 2C sums per CTA, its groups added in order
  float* row = a.part + (size_t)blockIdx.x * 4 * a.C;
  for (int i = threadIdx.x; i < 2 * a.C; i += kThreads) {
    double v = 0.0;
#pragma unroll
    for (int g = 0; g < G; ++g) v += sums[g * 2 * a.C + i];
    put_partial(row, a.C, i, v);
  }
}

// ------------------------------------------------------------------ host side

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

// What a call has chosen so far, and what it left to report.
struct Call {
  NormArgs n;
  int sms;
  cudaStream_t st;
  int rows = 0;
  cudaError_t err = cudaSuccess;
};

// Runs form F if its tiles fit: NC channels per row of lanes, three stages (two per group where
// rows are copied by their own lanes); `least` tiles per SM, or the caller tries a narrower form.
template <typename F, bool BWD>
bool try_form(Call& call, int least) {
  using T = typename F::T;
  const NormArgs& n = call.n;
  if (n.C > F::kRows * F::NC) return false;
  RingArgs a{};
  a.boxes = (n.C + 255) / 256;
  // an even number of rows: a box lands on 128 bytes, and a row may have 64
  a.box_rows = ((n.C + a.boxes - 1) / a.boxes + 1) & ~1;
  const size_t rows = F::kTma ? (size_t)a.boxes * a.box_rows : n.C;
  auto up128 = [](size_t v) { return (v + 127) & ~size_t(127); };
  const size_t array = up128(rows * F::kPitch);
  const size_t stage = up128(array * (BWD ? 2 : 1) + (BWD && F::kTma ? 8 * F::kPts : 0));
  const size_t tail = ring_tail<F, BWD>(n.C) + 128;
  int stages = (int)std::min<size_t>(kMaxStages, (kRingSmem - tail) / stage);
  // A stage stays with one group, whose warps then wait for each of its phases in order: were it to
  // go from group to group, a fast one could be two phases ahead, which a wait for a parity cannot
  // tell from none (13 stages and 4 groups: it may take tile 3 for tile 29).
  // Of rows copied by their own lanes at most four tiles are in flight.
  stages = (F::kTma ? stages / F::G : std::min(stages / F::G, 4)) * F::G;
  if (stages < (F::kTma ? 3 : 2 * F::G)) return false;
  a.tiles_per_plane = (int)((n.npts + F::kPts - 1) / F::kPts);
  a.tiles = (long long)n.B * a.tiles_per_plane;
  if (a.tiles < (long long)least * call.sms) return false;
  a.dout_off = (int)array;
  a.stat_off = (int)(2 * array);
  a.stage_bytes = (int)stage;
  a.stages = stages;
  a.B = n.B;
  a.C = n.C;
  a.npts = (int)n.npts;
  a.x = n.x;
  a.dout = n.dout;
  a.gain = n.gain;
  a.bias = n.bias;
  a.eps = n.eps;
  a.out = BWD ? n.dx : n.out;
  a.stats = n.stats;
  a.stats_in = n.stats;
  a.part = n.dgain || n.dbias ? n.part : nullptr;
  const int grid = (int)std::min<long long>(call.sms, a.tiles);
  const size_t smem = (size_t)stages * stage + tail;
  const bool bf16 = sizeof(T) == 2;
  call.rows = grid;
  CUtensorMap mx{}, md{};
  if (F::kTma && (!field_map(&mx, bf16, n.x, a, F::kPts) || (BWD && !field_map(&md, bf16, n.dout, a, F::kPts)))) {
    call.err = cudaErrorInvalidValue;
    return true;
  }
  auto run = [&](auto k, auto... maps) {
    // the same limit in every call: another thread may be between its own two calls here
    cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kRingSmem);
    if (e != cudaSuccess) return e;
    k<<<grid, kThreads, smem, call.st>>>(maps..., a);
    count_launch();
    return cudaGetLastError();
  };
  auto launch = [&](auto form) {
    using G = decltype(form);
    if constexpr (BWD) return run(norm_ring_bwd_kernel<G>, mx, md);
    else return run(norm_ring_fwd_kernel<G>, mx);
  };
  if constexpr (F::kTma) {
    if (n.C == F::kRows * F::NC) {
      call.err = launch(typename F::Filled{});
      return true;
    }
  }
  call.err = launch(F{});
  return true;
}

// The forms of either pass, few channels first.  A form has at most 32 registers of packed values;
// of those that hold the channels the first ones have the longer rows (runs of HBM) and the
// smaller groups (cheaper barriers).
template <typename T, int GRAN, bool BWD>
bool run_forms(Call& c) {
  constexpr int v16 = 16 / (int)sizeof(T), v8 = 8 / (int)sizeof(T);
  for (int least = 2; least >= 0; least -= 2) {
    if constexpr (!BWD) {
      if (least && (try_form<Form<T, v16, 32, 1, 8, GRAN>, BWD>(c, least) || try_form<Form<T, v16, 16, 1, 8, GRAN>, BWD>(c, least) ||
                    try_form<Form<T, v16, 16, 2, 8, GRAN>, BWD>(c, least) || try_form<Form<T, v16, 16, 4, 8, GRAN>, BWD>(c, least) ||
                    try_form<Form<T, v16, 16, 8, 8, GRAN>, BWD>(c, least)))
        return true;
      if (try_form<Form<T, v8, 16, 8, 4, GRAN>, BWD>(c, least) || try_form<Form<T, v8, 16, 8, 16, GRAN>, BWD>(c, least) ||
          try_form<Form<T, v8, 16, 16, 16, GRAN>, BWD>(c, least) || try_form<Form<T, v8, 8, 16, 16, GRAN>, BWD>(c, least))
        return true;
    } else {
      if (least && (try_form<Form<T, v8, 32, 1, 8, GRAN>, BWD>(c, least) || try_form<Form<T, v8, 16, 1, 8, GRAN>, BWD>(c, least) ||
                    try_form<Form<T, v8, 16, 2, 8, GRAN>, BWD>(c, least) || try_form<Form<T, v8, 16, 4, 8, GRAN>, BWD>(c, least)))
        return true;
      if (try_form<Form<T, v8, 16, 8, 4, GRAN>, BWD>(c, least) || try_form<Form<T, v8, 16, 8, 8, GRAN>, BWD>(c, least) ||
          try_form<Form<T, v8, 16, 16, 8, GRAN>, BWD>(c, least) || try_form<Form<T, v8, 8, 16, 8, GRAN>, BWD>(c, least))
        return true;
    }
  }
  return false;
}

template <typename T, int GRAN>
bool run_pass(Call& c, bool bwd) {
  return bwd ? run_forms<T, GRAN, true>(c) : run_forms<T, GRAN, false>(c);
}

// The widest of 16, 4 and 2 bytes that every plane starts on.
int granule(const NormArgs& n, int es) {
  int gran = 16;
  for (const void* q : {n.x, (const void*)n.out, n.dout, (const void*)n.dx})
    while (n.npts * es % gran || reinterpret_cast<uintptr_t>(q) % gran) gran >>= 1;
  if (gran == 16 && reinterpret_cast<uintptr_t>(n.stats) % 16) gran = 8;
  return gran == 8 ? 4 : gran;
}

}  // namespace

bool launch_norm_ring(bool bf16, const NormArgs& n, bool bwd, int sms, cudaStream_t st, int* rows, cudaError_t* err) {
  if (n.npts < 64) return false;
  Call c{n, sms, st};
  const int gran = granule(n, bf16 ? 2 : 4);
  bool ran;
  if (bf16) {
    ran = gran == 16 ? run_pass<__nv_bfloat16, 16>(c, bwd)
          : gran == 4 ? run_pass<__nv_bfloat16, 4>(c, bwd) : run_pass<__nv_bfloat16, 2>(c, bwd);
  } else {
    ran = gran == 16 ? run_pass<float, 16>(c, bwd) : run_pass<float, 4>(c, bwd);
  }
  *rows = c.rows;
  *err = c.err;
  return ran;
}

int take_norm_status() {
  int v = 0, z = 0;
  cudaMemcpyFromSymbol(&v, g_device_status, sizeof(int));
  if (v) cudaMemcpyToSymbol(g_device_status, &z, sizeof(int));
  return v;
}

}  // namespace disco
