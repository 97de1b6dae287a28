// The orthogonalised update of weights: Newton-Schulz products.
//
// For each (rows x cols) matrix U of a call (transposed if rows > cols, so that R <= L):
//   X = U / (|U|_F + eps), then `steps` times
//   A = X X^T,  B = a I + b A + c A A,  X <- B X
// which is the odd polynomial a s + b s^3 + c s^5 on each singular value s.
//
// Waits.  Every wait on an mbarrier is bounded.  After one that ran out a CTA waits and multiplies no
// more, still reaches every barrier of its cluster, lets what is in flight land and stores nothing; the
// others of its cluster store nothing either, and in a chain of kernels a word in the workspace tells
// the later ones, so that no weight is overwritten from void products.
//
// Three forms, by R alone unless the columns do not fit:
//   up to 32 rows      one launch, fp32 on the CUDA cores, a cluster of CTAs per matrix (of 32 rows up to
//                      4376 columns; longer ones take the next forms);
//   33 to 128 rows     one launch, tensor cores, X in shared memory for all steps, a cluster per matrix;
//   more               a chain of tiled products on tensor cores, operands in global memory (L2).
// Measured in fp32 (a call's time on the GPU): 4 x 12 in 6.7 us, 32 x 96 in 18.4, 64 x 192 in 34, eight 128 x 576 in 63,
// 256 x 2304 in 142, four 512 x 4608 in 387, 1024 x 9216 in 517, 32 x 9216 in 185.
//
// Numbers of the tensor-core forms.  A small singular value is multiplied by `a` in every step, and a
// rounding error of X in its direction with it: an X rounded to 8 or 11 bits would leave the weak
// directions of an update wrong by per cents.  So every matrix is kept as an fp16 pair hi + lo (22
// bits) under a power-of-two scale, and a product takes three MMAs, hi hi + hi lo + lo hi; what is
// left out, lo lo, is below 2^-22.  bf16 tensors get the same: with A and B from their hi parts alone
// matrices of a few rows came out 4e-3 off, twice what their own rounding leaves.  The two small
// products go into an accumulator of their own.  The tensor core cuts what it adds to an accumulator
// instead of rounding it (chains of 512 values left a 1024 x 9216 result 3.5e-5 off, 8 times fp32's
// error), so the large product is taken out and added in registers every 64 values, or spread over
// three or four accumulators (192 values in a chain at most).  Scales: X by 2^12, A by 2^11, B by 2^9,
// so that |X| <= 16, |A| <= 32, |B| <= 128 stay finite in fp16; lo by 2^11 more, which puts it at hi's
// size, so that it keeps its bits for entries far below the largest.
#include <cuda.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "common.cuh"
#include "kernels.h"
#include "muon.h"
#include "tc_common.cuh"

namespace disco {
namespace {

constexpr float kSx = 4096.0f, kSa = 2048.0f, kSb = 512.0f, kSl = 2048.0f;
constexpr int kTile = 128;       // a CTA's rows of a product's tile, and its share of the operands
constexpr int kBk = 64;          // K values per stage: one 128-byte swizzle row of fp16
constexpr int kMaxSplits = 8;    // of the K range of a product
constexpr int kLeastJoin = 8;      // chunks of a product that a cluster of single CTAs shares, at least
constexpr int kStages = 3;
constexpr uint32_t kOperand = kTile * 128;   // one [128][64] fp16 operand tile, bytes
constexpr uint32_t kStageBytes = 4 * kOperand;
constexpr int kDrainWarps = 16;
constexpr int kProductThreads = (kDrainWarps + 2) * 32;
constexpr int kTensors = 64;     // tensors of one set of launches (pointers travel as arguments)
constexpr int kNormBlocks = 256;  // partial sums of squares per matrix, at most

struct Pointers {
  const void* in[kTensors];
  const void* w[kTensors];
  const float* m[kTensors];
  void* out[kTensors];
  float* m_out[kTensors];
};

struct Shape {
  int groups, rows, cols;
  int R, L, Rp, Lp;  // iterated matrix (R <= L) and its padded sides, multiples of `tile`
  int tile;          // side of a product's tile: 256 (a pair of CTAs) or 128 (one CTA)
  bool tr;           // iterated on the transposed matrix
  int nm;            // matrices
};

struct Rule {
  bool step, nesterov;
  float momentum, keep, rate;
};

// Programmatic dependent launch: the next kernel of a chain may be brought up while this one runs,
// and waits here for the results of the one before it.
__device__ __forceinline__ void wait_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// hi + lo / kSl = v to 22 bits (v within fp16's range).
__device__ __forceinline__ void split(float v, __half& hi, __half& lo) {
  hi = __float2half_rn(v);
  lo = __float2half_rn((v - __half2float(hi)) * kSl);
}

__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
  for (int m = 16; m; m >>= 1) v += __shfl_xor_sync(~0u, v, m);
  return v;
}

// kWide values from an address on their own alignment, by one load where it is wide enough.
constexpr int kWide = 8;
template <typename T>
__device__ __forceinline__ void load_wide(const T* p, int n, float (&v)[kWide]) {
  if (n == kWide && reinterpret_cast<uintptr_t>(p) % 16 == 0) {
    alignas(16) T q[kWide];
#pragma unroll
    for (int i = 0; i < kWide * (int)sizeof(T) / 16; ++i)
      reinterpret_cast<uint4*>(q)[i] = reinterpret_cast<const uint4*>(p)[i];
#pragma unroll
    for (int i = 0; i < kWide; ++i) v[i] = to_f32(q[i]);
  } else {
#pragma unroll
    for (int i = 0; i < kWide; ++i) v[i] = i < n ? to_f32(p[i]) : 0.0f;
  }
}
template <typename T>
__device__ __forceinline__ void store_wide(T* p, int n, const float (&v)[kWide]) {
  if (n == kWide && reinterpret_cast<uintptr_t>(p) % 16 == 0) {
    alignas(16) T q[kWide];
#pragma unroll
    for (int i = 0; i < kWide; ++i) q[i] = from_f32<T>(v[i]);
#pragma unroll
    for (int i = 0; i < kWide * (int)sizeof(T) / 16; ++i)
      reinterpret_cast<uint4*>(p)[i] = reinterpret_cast<const uint4*>(q)[i];
  } else {
#pragma unroll
    for (int i = 0; i < kWide; ++i)
      if (i < n) p[i] = from_f32<T>(v[i]);
  }
}

// The update itself from the gradient u and the momentum m before it (after it: m_new).
__device__ __forceinline__ float new_momentum(const Rule& r, float u, float m) { return fmaf(r.momentum, m, u); }
__device__ __forceinline__ float update_of(const Rule& r, float u, float m_new) {
  return r.nesterov ? fmaf(r.momentum, m_new, u) : m_new;
}

// What is stored of a result: the new weight from the old one, or the result itself.
__device__ __forceinline__ float result_of(const Rule& r, float w, float x) {
  return r.step ? fmaf(r.keep, w, -r.rate * x) : x;
}

// Sums of squares of a slice of each matrix; for a whole step the momentum is updated on the way.
// fp64: no update is too large or too small for its square.  *fail: the chain's failure word.
template <typename T>
__global__ void __launch_bounds__(256) ns_norm_kernel(const __grid_constant__ Pointers p, Shape s, Rule r,
                                                      double* __restrict__ part, int* fail) {
  __shared__ double warps[8];
  if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) *fail = 0;
  let_next_start();
  const int mi = blockIdx.y, t = mi / s.groups, g = mi % s.groups;
  const size_t n = (size_t)s.rows * s.cols, base = g * n;
  const T* in = static_cast<const T*>(p.in[t]) + base;
  const float* m = r.step ? p.m[t] + base : nullptr;
  float* mo = r.step ? p.m_out[t] + base : nullptr;
  double sum[2] = {0.0, 0.0};
  const size_t stride = (size_t)gridDim.x * 256 * kWide;
#pragma unroll 2
  for (size_t i = ((size_t)blockIdx.x * 256 + threadIdx.x) * kWide; i < n; i += stride) {
    const int here = (int)(n - i < kWide ? n - i : kWide);
    float u[kWide];
    load_wide(in + i, here, u);
    if (r.step) {
      float v[kWide];
      load_wide(m + i, here, v);
#pragma unroll
      for (int k = 0; k < kWide; ++k) v[k] = new_momentum(r, u[k], v[k]);
      store_wide(mo + i, here, v);
#pragma unroll
      for (int k = 0; k < kWide; ++k) u[k] = update_of(r, u[k], v[k]);
    }
#pragma unroll
    for (int k = 0; k < kWide; ++k) sum[k & 1] = fma((double)u[k], (double)u[k], sum[k & 1]);
  }
  const double all = warp_sum(sum[0] + sum[1]);
  if ((threadIdx.x & 31) == 0) warps[threadIdx.x >> 5] = all;
  __syncthreads();
  if (threadIdx.x == 0) {
    double v = 0.0;
    for (int k = 0; k < 8; ++k) v += warps[k];
    part[(size_t)mi * gridDim.x + blockIdx.x] = v;
  }
}

// X = U / (|U|_F + eps) as hi and lo planes [2][nm][Rp][Lp], zero in the padding: a 64 x 64 tile a CTA.
template <typename T>
__global__ void __launch_bounds__(256) ns_load_kernel(const __grid_constant__ Pointers p, Shape s, Rule r, double eps,
                                                      const double* __restrict__ part, int parts,
                                                      __half* __restrict__ x) {
  __shared__ float tile[64][65];
  __shared__ float scale;
  const int mi = blockIdx.z, t = mi / s.groups, g = mi % s.groups;
  let_next_start();
  wait_previous();
  if (threadIdx.x < 32) {
    double v = 0.0;
    for (int k = threadIdx.x; k < parts; k += 32) v += part[(size_t)mi * parts + k];
    v = warp_sum(v);
    if (threadIdx.x == 0) scale = (float)((double)kSx / (sqrt(v) + eps));
  }
  const size_t base = (size_t)g * s.rows * s.cols;
  const T* in = static_cast<const T*>(p.in[t]) + base;
  const float* mo = r.step ? p.m_out[t] + base : nullptr;
  const int l0 = blockIdx.x * 64, r0 = blockIdx.y * 64;
  const int x8 = threadIdx.x % 8 * kWide, y = threadIdx.x / 8;
  // a row of the tile is read along the tensor's columns
#pragma unroll
  for (int k = y; k < 64; k += 32) {
    const int row = (s.tr ? l0 : r0) + k, col = (s.tr ? r0 : l0) + x8;
    const int here = row < s.rows ? max(0, min(kWide, s.cols - col)) : 0;
    float u[kWide] = {};
    if (here > 0) {
      const size_t i = (size_t)row * s.cols + col;
      load_wide(in + i, here, u);
      if (r.step) {
        float m[kWide];
        load_wide(mo + i, here, m);
#pragma unroll
        for (int e = 0; e < kWide; ++e) u[e] = update_of(r, u[e], m[e]);
      }
    }
#pragma unroll
    for (int e = 0; e < kWide; ++e) tile[k][x8 + e] = u[e];
  }
  __syncthreads();
  const size_t plane = (size_t)s.nm * s.Rp * s.Lp;
#pragma unroll
  for (int k = y; k < 64; k += 32) {
    alignas(16) __half h[kWide], l[kWide];
#pragma unroll
    for (int e = 0; e < kWide; ++e) split((s.tr ? tile[x8 + e][k] : tile[k][x8 + e]) * scale, h[e], l[e]);
    const size_t at = ((size_t)mi * s.Rp + r0 + k) * s.Lp + l0 + x8;
    *reinterpret_cast<uint4*>(x + at) = *reinterpret_cast<const uint4*>(h);
    *reinterpret_cast<uint4*>(x + plane + at) = *reinterpret_cast<const uint4*>(l);
  }
}

// ------------------------------------------------------------------ the products

enum Product { kSymmetric, kUpdate, kFinal };
enum Team { kAlone, kPair, kJoined };  // who makes a tile: one CTA, a pair, a cluster over parts of K

// What becomes of the entries of a symmetric product: A from those of X X^T (am null), or
// B = a I + b A + c A A from those of A A.
struct Becomes {
  float a, b, c;
  const __half* am;
};

struct ProductArgs {
  Shape s;
  int tm, tn, S, chunks;  // tiles along M and N, splits along K, K chunks in all
  bool upper;             // P is kept on and above the diagonal only
  float* part;            // kSymmetric, S > 1: [S][nm][Rp][Rp]
  Becomes f;              // kSymmetric, S = 1: what the product becomes, into dst
  __half* dst;            // kUpdate: the next X
  int* fail;              // set when a wait of the chain ran out
  unsigned long long hold_ns;  // self test: nothing is loaded, and waits are given up after this
  Rule r;
};

__device__ __forceinline__ uint8_t* align1024(uint8_t* p) {
  return reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(p) + 1023) & ~uintptr_t(1023));
}

// Instruction descriptor: fp16 x fp16 -> fp32, M x N, A and B major modes.
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N, bool a_mn_major, bool b_mn_major) {
  return (1u << 4) | ((a_mn_major ? 1u : 0u) << 15) | ((b_mn_major ? 1u : 0u) << 16) | ((uint32_t)(N >> 3) << 17) |
         ((uint32_t)(M >> 4) << 24);
}

// 8 values as 16 bytes of hi and of lo.
__device__ __forceinline__ void split8(const float (&v)[8], uint4& hi, uint4& lo) {
  alignas(16) __half2 h[4], l[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    h[i] = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
    const float2 f = __half22float2(h[i]);
    l[i] = __floats2half2_rn((v[2 * i] - f.x) * kSl, (v[2 * i + 1] - f.y) * kSl);
  }
  hi = *reinterpret_cast<const uint4*>(h);
  lo = *reinterpret_cast<const uint4*>(l);
}
__device__ __forceinline__ void widen8(uint4 hi, float (&v)[8]) {
  const __half2* h = reinterpret_cast<const __half2*>(&hi);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 x = __half22float2(h[i]);
    v[2 * i] = x.x;
    v[2 * i + 1] = x.y;
  }
}
__device__ __forceinline__ void join8(uint4 hi, uint4 lo, float (&v)[8]) {
  float w[8];
  widen8(hi, v);
  widen8(lo, w);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = fmaf(w[i], 1.0f / kSl, v[i]);
}
// 8 entries of a row of a symmetric product, scaled as the next operand; `diag`: which of them lies
// on the diagonal, if any.
__device__ __forceinline__ void become(const Becomes& f, size_t plane, size_t at, int diag, float (&v)[8]) {
  if (!f.am) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] *= kSa / (kSx * kSx);
    return;
  }
  float x[8];
  join8(*reinterpret_cast<const uint4*>(f.am + at), *reinterpret_cast<const uint4*>(f.am + plane + at), x);
#pragma unroll
  for (int i = 0; i < 8; ++i)
    v[i] = fmaf(f.c * (kSb / (kSa * kSa)), v[i], fmaf(f.b * (kSb / kSa), x[i], i == diag ? f.a * kSb : 0.0f));
}

// One tile of a product of hi + lo matrices: D = P P^T (kSymmetric, tiles on and above the diagonal
// only) or D = P Q (kUpdate, kFinal; Q is read as an MN-major operand).  P is X, or one of the
// symmetric matrices A and B, of which only the tiles on and above the diagonal are kept (`upper`): a
// chunk below it is loaded from its mirror image and read as an MN-major operand (writing the mirror
// images instead cost 3 to 5 us a product).
//
// PAIR: two CTAs (cta_group::2) make a 256 x 256 tile.  Each brings 128 rows of P and 128 columns of Q
// and gets 128 rows of D, so that 64 KB from L2 feed 1536 cycles of MMA; one CTA with a 128 x 128 tile
// needs 64 KB for 768, more than L2 gives when all SMs ask (1024 x 9216: 2.4x slower).  Below one
// tile for every pair latency counts instead, and one CTA makes a 128 x 128 tile, or a cluster of S
// CTAs does, each over its part of K: then each adds a band of rows of all their sums, in an order of
// its own that never changes, and writes it.  (Pairs split only symmetric products, through partial sums in global memory.)
//
// Warp 16 streams the four operand tiles of each K chunk by TMA, all counted on the first CTA's
// barrier; lane 0 of the first CTA's warp 17 issues the MMAs for both; warps 0..15 of both CTAs add
// the chunk's large product to their sums (TMEM lane = row of the tile, a quarter of the columns a
// warp) while the MMAs of its small products run.
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ uint32_t at_rank(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ float4 ld_remote(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
// The same box load, counted on a barrier of either CTA of the pair.
__device__ __forceinline__ void pair_load_3d(void* dst, const CUtensorMap* map, uint32_t bar, int c0, int c1, int c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, "
      "%5}], [%2];" ::"r"(tc::smem_u32(dst)),
      "l"(map), "r"(bar), "r"(c0), "r"(c1), "r"(c2)
      : "memory");
}
__device__ __forceinline__ void pair_mma(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                         uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Arrives on `bar` of both CTAs once every MMA this thread has issued is done.
__device__ __forceinline__ void pair_commit(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
          tc::smem_u32(bar)),
      "h"((uint16_t)3)
      : "memory");
}
__device__ __forceinline__ void st_remote(uint32_t addr, int v) {
  asm volatile("st.shared::cluster.b32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
// Sets `bad` of this CTA, and of all S of its cluster.
__device__ __forceinline__ void mark_bad(int* bad, int S) {
  *reinterpret_cast<volatile int*>(bad) = 1;
  for (int k = 0; S > 1 && k < S; ++k) st_remote(at_rank(tc::smem_u32(bad), k), 1);
}
// Arrives on a barrier of either CTA.  What it orders is this warp's reads of TMEM, which are
// complete (wait::ld), and no memory: a release over the cluster would cost a fence a chunk.
__device__ __forceinline__ void arrive_remote(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

template <typename T, Product MODE, Team TEAM>
__global__ void __launch_bounds__(kProductThreads, 1)
    ns_product_kernel(const __grid_constant__ CUtensorMap map_p, const __grid_constant__ CUtensorMap map_q,
                      const __grid_constant__ Pointers ptr, const __grid_constant__ ProductArgs a) {
  constexpr bool PAIR = TEAM == kPair, joined = TEAM == kJoined;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align1024(smem_raw);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + kStages * kStageBytes);
  uint64_t* empty = full + kStages;
  uint64_t* tfull = empty + kStages;  // the chunk's large product is in TMEM
  uint64_t* tempty = tfull + 1;       // and every CTA has read it
  uint64_t* done = tempty + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);
  int* bad = reinterpret_cast<int*>(tmem_slot + 1);  // a wait ran out here, in the cluster that shares K or before
  constexpr bool kMn = MODE != kSymmetric;
  constexpr int kCtas = PAIR ? 2 : 1, kSide = kCtas * kTile, kCols = kSide / 4;  // columns of a warp
  const Shape& s = a.s;
  const uint32_t rank = PAIR ? cluster_rank() : 0;  // of the pair
  const int job = (int)blockIdx.x / kCtas;
  int tile = job / a.S, bm = 0, bn = 0;
  const int split_k = job % a.S;                    // and the rank of a joined CTA in its cluster
  if (MODE == kSymmetric) {
    while (tile >= a.tn - bm) tile -= a.tn - bm++;
    bn = bm + tile;
  } else {
    bm = tile % a.tm;
    bn = tile / a.tm;
  }
  const int m0 = bm * kSide + (int)rank * kTile, n0 = bn * kSide, qn = n0 + (int)rank * kTile;
  const int mi = blockIdx.y;
  const int k_lo = a.chunks * split_k / a.S, k_hi = a.chunks * (split_k + 1) / a.S;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // whether a chunk of P (of Q) comes as the mirror image, and is then MN-major like Q of an update
  auto p_mn = [&](int k) { return a.upper && k * kBk / kSide < bm; };
  auto q_mn = [&](int k) { return kMn || (a.upper && k * kBk / kSide < bn); };
  auto all_sync = [] {
    if constexpr (PAIR || joined) cluster_sync();
    else __syncthreads();
  };

  if (threadIdx.x == 0) {
    tc::prefetch_map(&map_p);
    tc::prefetch_map(&map_q);
    for (int i = 0; i < kStages; ++i) {
      tc::mbar_init(&full[i], 1);
      tc::mbar_init(&empty[i], 1);
    }
    tc::mbar_init(tfull, 1);
    tc::mbar_init(tempty, kCtas * kDrainWarps);
    tc::mbar_init(done, 1);
    tc::fence_barrier_init();
    *bad = 0;
  }
  if (warp == kDrainWarps + 1) {
    if constexpr (PAIR) {
      asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(tc::smem_u32(tmem_slot)),
                   "r"(2u * kSide)
                   : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    } else {
      tc::tmem_alloc(tmem_slot, 2 * kSide);
      tc::tmem_relinquish();
    }
  }
  let_next_start();
  tc::fence_before_sync();
  all_sync();
  tc::fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  wait_previous();
  // whether no wait ran out before this kernel; the loads do not wait for the answer (0.5 us a product)
  auto sound = [&] { return *reinterpret_cast<const volatile int*>(a.fail) == 0; };
  bool ok = true;
  const unsigned long long limit = a.hold_ns ? a.hold_ns : tc::kWaitNs;
  auto wait = [&](uint64_t* bar, uint32_t parity) { return tc::mbar_wait(bar, parity, limit); };

  if (warp == kDrainWarps && lane == 0) {
    for (int k = a.hold_ns ? k_hi : k_lo; k < k_hi; ++k) {
      const int i = k - k_lo, st = i % kStages;
      if (i == kStages) ok = sound();
      ok = ok && (i < kStages || wait(&empty[st], ((i / kStages) & 1) ^ 1));
      if (!ok) break;
      uint8_t* base = smem + st * kStageBytes;
      const uint32_t bar = PAIR ? at_rank(tc::smem_u32(&full[st]), 0) : 0;
      if (rank == 0) tc::mbar_arrive_expect_tx(&full[st], kCtas * kStageBytes);
      auto load = [&](uint8_t* dst, const CUtensorMap* map, int c0, int c1, int z) {
        if constexpr (PAIR) pair_load_3d(dst, map, bar, c0, c1, z);
        else tc::tma_load_3d(dst, map, &full[st], c0, c1, z);
      };
#pragma unroll
      for (int pl = 0; pl < 2; ++pl) {
        const int z = pl * s.nm + mi;
        uint8_t* pp = base + pl * kOperand;
        uint8_t* qq = base + (2 + pl) * kOperand;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (p_mn(k)) load(pp + h * (kOperand / 2), &map_p, m0 + 64 * h, k * kBk, z);
          else load(pp + h * (kOperand / 2), &map_p, k * kBk, m0 + 64 * h, z);
          if (q_mn(k)) load(qq + h * (kOperand / 2), &map_q, qn + 64 * h, k * kBk, z);
          else load(qq + h * (kOperand / 2), &map_q, k * kBk, qn + 64 * h, z);
        }
      }
    }
  } else if (warp == kDrainWarps + 1 && lane == 0 && rank == 0) {
    auto commit = [](uint64_t* bar) {
      if constexpr (PAIR) pair_commit(bar);
      else tc::mma_commit(bar);
    };
    ok = sound();
    for (int k = k_lo; k < k_hi; ++k) {
      const int i = k - k_lo, st = i % kStages;
      ok = ok && wait(&full[st], (i / kStages) & 1) && (i == 0 || wait(tempty, (i & 1) ^ 1));
      if (!ok) break;
      tc::fence_after_sync();
      const uint32_t p0 = tc::smem_u32(smem + st * kStageBytes), q0 = p0 + 2 * kOperand;
      const bool pm = p_mn(k), qm = q_mn(k);
      const uint32_t idesc = idesc_f16(kSide, kSide, pm, qm);
      auto operand = [](uint32_t base, bool mn, int kk) {
        return mn ? tc::desc_sw128(base + kk * 2048, kOperand / 2, 1024) : tc::desc_sw128(base + kk * 32, 16, 1024);
      };
      auto mma = [&](uint32_t d, int p_plane, int q_plane, int kk, uint32_t more) {
        const uint64_t x = operand(p0 + p_plane * kOperand, pm, kk), y = operand(q0 + q_plane * kOperand, qm, kk);
        if constexpr (PAIR) pair_mma(d, x, y, idesc, more);
        else tc::mma_bf16(d, x, y, idesc, more);
      };
#pragma unroll
      for (int kk = 0; kk < kBk / 16; ++kk) mma(tmem, 0, 0, kk, kk != 0);
      commit(tfull);
#pragma unroll
      for (int kk = 0; kk < kBk / 16; ++kk) {
        mma(tmem + kSide, 0, 1, kk, (i | kk) != 0);
        mma(tmem + kSide, 1, 0, kk, 1);
      }
      commit(&empty[st]);
    }
    commit(done);
  }
  __syncwarp();
  // The tile goes through the operand buffers, which are free: 128 rows of kSide fp32 values, the
  // 16-byte blocks of a row exchanged by the row's last bits.  What is made of it then runs in
  // short loops: unrolled over a thread's registers the code came cold from L2 and cost 8 us.
  constexpr uint32_t kRowBytes = kSide * 4;
  auto block_of = [&](int r, int block) {
    return reinterpret_cast<float4*>(smem + r * kRowBytes + (((uint32_t)block ^ ((uint32_t)r & 7u)) << 4));
  };
  if (warp < kDrainWarps) {
    const int quarter = (warp & 3) * 32, c0 = (warp >> 2) * kCols;
    const uint32_t tw = tmem + ((uint32_t)quarter << 16) + c0;
    const uint32_t release = PAIR ? at_rank(tc::smem_u32(tempty), 0) : 0;
    float acc[kCols];
#pragma unroll
    for (int i = 0; i < kCols; ++i) acc[i] = 0.0f;
    ok = sound();
    for (int i = 0; i < k_hi - k_lo && ok; ++i) {
      ok = __all_sync(~0u, wait(tfull, i & 1));
      if (!ok) break;
      tc::fence_after_sync();
#pragma unroll
      for (int h = 0; h < kCols; h += 32) {
        uint32_t v[32];
        tc::tmem_ld_chunks<2>(tw + h, v);
        if (h + 32 == kCols) {
          tc::fence_before_sync();
          __syncwarp();
          if (lane == 0) {
            if constexpr (PAIR) arrive_remote(release);
            else tc::mbar_arrive(tempty);
          }
        }
#pragma unroll
        for (int c = 0; c < 32; ++c) acc[h + c] += __uint_as_float(v[c]);
      }
    }
    ok = ok && __all_sync(~0u, wait(done, 0));
    if (ok) {  // so all chunks were loaded and multiplied, and the operand buffers are free
      tc::fence_after_sync();
#pragma unroll
      for (int c = 0; c < kCols; c += 16) {
        float v[16];
        tc::tmem_ld16(tw + kSide + c, v);
#pragma unroll
        for (int i = 0; i < 16; i += 4)
          *block_of(quarter + lane, (c0 + c + i) / 4) =
              make_float4(fmaf(v[i], 1.0f / kSl, acc[c + i]), fmaf(v[i + 1], 1.0f / kSl, acc[c + i + 1]),
                          fmaf(v[i + 2], 1.0f / kSl, acc[c + i + 2]), fmaf(v[i + 3], 1.0f / kSl, acc[c + i + 3]));
      }
      tc::fence_before_sync();
    }
  }
  if (!ok) mark_bad(bad, joined ? a.S : 1);
  if constexpr (joined) cluster_sync();  // the sums of all CTAs of the cluster are in their buffers
  else __syncthreads();
  const bool store = *reinterpret_cast<volatile int*>(bad) == 0;
  // 16 bytes of the tile, over all parts of K
  auto sum_of = [&](int r, int block) {
    float4 v = *block_of(r, block);
    if constexpr (joined) {  // from itself on: all would ask the same CTA at a time otherwise
      const uint32_t addr = tc::smem_u32(block_of(r, block));
      float4 x[kMaxSplits];
#pragma unroll
      for (int k = 1; k < kMaxSplits; ++k)
        if (k < a.S) x[k] = ld_remote(at_rank(addr, (split_k + k) & (a.S - 1)));
#pragma unroll
      for (int k = 1; k < kMaxSplits; ++k) {
        if (k < a.S) {
          v.x += x[k].x;
          v.y += x[k].y;
          v.z += x[k].z;
          v.w += x[k].w;
        }
      }
    }
    return v;
  };
  if (warp < kDrainWarps && store) {
    const size_t pa = (size_t)s.nm * s.Rp * s.Rp, px = (size_t)s.nm * s.Rp * s.Lp;
    const size_t tensor = (size_t)(mi % s.groups) * s.rows * s.cols;
    if (PAIR && MODE == kSymmetric && a.S > 1) {
#pragma unroll 2
      for (int r = warp; r < kTile; r += kDrainWarps) {  // a warp takes a row, a lane 4 columns of each 128
        float* dst = a.part + (size_t)split_k * pa + ((size_t)mi * s.Rp + m0 + r) * s.Rp + n0 + lane * 4;
#pragma unroll
        for (int h = 0; h < kCtas; ++h) *reinterpret_cast<float4*>(dst + 128 * h) = *block_of(r, lane + 32 * h);
      }
    } else if (!(MODE == kFinal && s.tr)) {
      constexpr int kLanes = kSide / 8;  // lanes of a row, 8 columns each
      const int lr = lane % kLanes;
      const int r_lo = joined ? kTile * split_k / a.S : 0, r_hi = joined ? kTile * (split_k + 1) / a.S : kTile;
#pragma unroll 2
      for (int r = r_lo + warp * (32 / kLanes) + lane / kLanes; r < r_hi; r += kDrainWarps * (32 / kLanes)) {
        const float4 x = sum_of(r, 2 * lr), y = sum_of(r, 2 * lr + 1);
        float v[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
        const int row = m0 + r, col = n0 + lr * 8;
        if constexpr (MODE == kSymmetric) {
          const size_t at = ((size_t)mi * s.Rp + row) * s.Rp + col;
          become(a.f, pa, at, row - col, v);
          uint4 hi, lo;
          split8(v, hi, lo);
          *reinterpret_cast<uint4*>(a.dst + at) = hi;
          *reinterpret_cast<uint4*>(a.dst + pa + at) = lo;
        } else if constexpr (MODE == kUpdate) {
          const size_t at = ((size_t)mi * s.Rp + row) * s.Lp + col;
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] *= 1.0f / kSb;
          uint4 hi, lo;
          split8(v, hi, lo);
          *reinterpret_cast<uint4*>(a.dst + at) = hi;
          *reinterpret_cast<uint4*>(a.dst + px + at) = lo;
        } else {
          const int here = row < s.R ? max(0, min(8, s.L - col)) : 0;
          if (here > 0) {
            const size_t at = tensor + (size_t)row * s.cols + col;
            float w[8] = {};
            if (a.r.step) load_wide(static_cast<const T*>(ptr.w[mi / s.groups]) + at, here, w);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = result_of(a.r, w[i], v[i] * (1.0f / (kSb * kSx)));
            store_wide(static_cast<T*>(ptr.out[mi / s.groups]) + at, here, v);
          }
        }
      }
    } else {
      // a warp takes 32 rows of 4 columns, of this CTA's share of the columns
      const int b_lo = joined ? kSide / 4 * split_k / a.S : 0, b_hi = joined ? kSide / 4 * (split_k + 1) / a.S : kSide / 4;
#pragma unroll 2
      for (int k = b_lo * 4 + warp; k < b_hi * 4; k += kDrainWarps) {
        const int r = k % 4 * 32 + lane, row = m0 + r, col = n0 + k / 4 * 4;
        const float4 x = sum_of(r, k / 4);
        const float v[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (row < s.R && col + i < s.L) {
            const size_t at = tensor + (size_t)(col + i) * s.cols + row;
            const float w = a.r.step ? to_f32(static_cast<const T*>(ptr.w[mi / s.groups])[at]) : 0.0f;
            static_cast<T*>(ptr.out[mi / s.groups])[at] = from_f32<T>(result_of(a.r, w, v[i] * (1.0f / (kSb * kSx))));
          }
        }
      }
    }
  }
  if (!store) {
    if (threadIdx.x == 0) *reinterpret_cast<volatile int*>(a.fail) = 1;
    tc::give_up();
  }
  // no CTA leaves before another's last arrival, MMA or read
  all_sync();
  if (warp == kDrainWarps + 1) {
    if constexpr (PAIR)
      asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(2u * kSide) : "memory");
    else tc::tmem_dealloc(tmem, 2 * kSide);
  }
}

// The next operand from the partial products of a symmetric product split along K, added in a fixed
// order: 64 x 64 entries a CTA, those of the tiles on and above the diagonal.
__global__ void __launch_bounds__(256) ns_reduce_kernel(const float* __restrict__ part, Shape s, int S, Becomes f,
                                                        __half* __restrict__ dst) {
  let_next_start();
  wait_previous();
  const int mi = blockIdx.z, bi = blockIdx.y, bj = blockIdx.x;
  if (bi * 64 / s.tile > bj * 64 / s.tile) return;
  const size_t plane = (size_t)s.nm * s.Rp * s.Rp, base = (size_t)mi * s.Rp * s.Rp;
  const int x = threadIdx.x % 8 * 8, y = threadIdx.x / 8;
#pragma unroll
  for (int r = y; r < 64; r += 32) {
    const int i = bi * 64 + r, j = bj * 64 + x;
    const size_t at = base + (size_t)i * s.Rp + j;
    float v[8] = {};
#pragma unroll 4
    for (int k = 0; k < S; ++k) {
#pragma unroll
      for (int e = 0; e < 8; e += 4) {
        const float4 p = *reinterpret_cast<const float4*>(part + k * plane + at + e);
        v[e] += p.x;
        v[e + 1] += p.y;
        v[e + 2] += p.z;
        v[e + 3] += p.w;
      }
    }
    become(f, plane, at, i - j, v);
    uint4 hi, lo;
    split8(v, hi, lo);
    *reinterpret_cast<uint4*>(dst + at) = hi;
    *reinterpret_cast<uint4*>(dst + plane + at) = lo;
  }
}

// ------------------------------------------------------------------ small matrices: one launch
//
// Matrices of up to 128 rows stay in shared memory for all steps.  A cluster of S CTAs takes one
// matrix, each CTA a run of 64-column chunks of X.  Per step every CTA adds its columns' share of
// X X^T, the shares are summed by blocks of columns (CTA q sums the q-th block of everybody's share)
// and each block goes to all CTAs; A A and B are formed by every CTA for itself, and B X for its
// own columns.  What bounds it is latency: 15 products that wait for one another, each a few
// hundred cycles of tensor core, and two cluster barriers a step.
//
// X chunk: [RP rows][64 columns] fp16, rows of 128 bytes in the 128-byte swizzle.  The same tile is
// the K-major operand of X X^T (K = columns) and the MN-major operand of B X (K = rows).  MMAs have
// M = 128; with RP = 64 rows 64..127 of an operand are whatever follows the tile, and the rows of the
// result they make are not read.

constexpr int kSmallThreads = 512;
constexpr int kSides = kSmallThreads / 128;    // warps that share 32 lanes of TMEM, each a run of columns
constexpr int kSmallMaxCluster = 8;
constexpr size_t kSmallSmem = 226 * 1024;      // of 227 KB
constexpr size_t kSmallLeast = 120 * 1024;     // more than half of an SM: one CTA (and its TMEM) per SM

struct SmallArgs {
  Shape s;
  Rule r;
  float a, b, c;
  double eps;
  int steps, S, nc, max_chunks;
  unsigned long long hold_ns;  // self test: the first CTA withholds its first product, and waits are given up after this
};

// Byte offsets of a CTA's shared memory.
struct SmallLayout {
  uint32_t xl, ah, al, recv, misc, total;
};
__host__ __device__ constexpr SmallLayout small_layout(int rp, int S, int max_chunks) {
  SmallLayout l{};
  const uint32_t chunk = rp * 128, a = (rp / 64) * chunk;
  l.xl = max_chunks * chunk;
  l.ah = 2 * l.xl;
  l.al = l.ah + a;
  l.recv = l.al + a;
  l.misc = l.recv + (S > 1 ? rp * rp * 4 : 0);
  l.total = l.misc + 1024 + (rp < 128 ? 8192 : 0);
  return l;
}

__device__ __forceinline__ uint32_t sw128(int row, int col_byte) {
  return (uint32_t)row * 128u + ((uint32_t)col_byte ^ (((uint32_t)row & 7u) << 4));
}
__device__ __forceinline__ void st_remote(uint32_t addr, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}
__device__ __forceinline__ void st_remote(uint32_t addr, double v) {
  asm volatile("st.shared::cluster.f64 [%0], %1;" ::"r"(addr), "d"(v) : "memory");
}
__device__ __forceinline__ void st_remote(uint32_t addr, uint4 v) {
  asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
               : "memory");
}
// Generic-proxy writes to shared memory of the whole cluster before later async-proxy reads.
__device__ __forceinline__ void fence_proxy_async_all() { asm volatile("fence.proxy.async;" ::: "memory"); }

// 8 fp32 values kept in the places of 8 hi and 8 lo halves, bit for bit.
__device__ __forceinline__ void bits8(const float (&v)[8], uint4& hi, uint4& lo) {
  uint32_t h[4], l[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t a = __float_as_uint(v[2 * i]), b = __float_as_uint(v[2 * i + 1]);
    h[i] = __byte_perm(a, b, 0x7632);
    l[i] = __byte_perm(a, b, 0x5410);
  }
  hi = make_uint4(h[0], h[1], h[2], h[3]);
  lo = make_uint4(l[0], l[1], l[2], l[3]);
}
__device__ __forceinline__ void unbits8(uint4 hi, uint4 lo, float (&v)[8]) {
  const uint32_t h[4] = {hi.x, hi.y, hi.z, hi.w}, l[4] = {lo.x, lo.y, lo.z, lo.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(__byte_perm(l[i], h[i], 0x5410));
    v[2 * i + 1] = __uint_as_float(__byte_perm(l[i], h[i], 0x7632));
  }
}

// 16 columns of a lane's row: the large product plus the small ones.
__device__ __forceinline__ void drain16(uint32_t main, uint32_t small, float (&v)[16]) {
  uint32_t r[16], e[16];
  tc::tmem_ld_chunks<1>(main, r);
  tc::tmem_ld_chunks<1>(small, e);
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = fmaf(__uint_as_float(e[i]), 1.0f / kSl, __uint_as_float(r[i]));
}

template <typename T, int RP>
__global__ void __launch_bounds__(kSmallThreads, 1)
    ns_small_kernel(const __grid_constant__ Pointers ptr, const __grid_constant__ SmallArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align1024(smem_raw);
  constexpr uint32_t kChunk = RP * 128;
  const SmallLayout lay = small_layout(RP, a.S, a.max_chunks);
  uint8_t *xh = smem, *xl = smem + lay.xl, *ah = smem + lay.ah, *al = smem + lay.al;
  float* recv = reinterpret_cast<float*>(smem + lay.recv);
  double* norms = reinterpret_cast<double*>(smem + lay.misc);  // [cluster]
  double* warps = norms + kSmallMaxCluster;                    // [16]
  uint64_t* done = reinterpret_cast<uint64_t*>(warps + kSmallThreads / 32);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);
  int* bad = reinterpret_cast<int*>(tmem_slot + 1);  // a wait ran out somewhere in the cluster
  const Shape& s = a.s;
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
  const int S = a.S, q = S > 1 ? (int)cluster_rank() : 0, mi = blockIdx.x / S;
  const int c_lo = a.nc * q / S, mine = a.nc * (q + 1) / S - c_lo;
  const int quarter = (warp & 3) * 32, side = warp >> 2;  // TMEM lanes and run of the columns
  const int row = quarter + lane;
  const bool live = quarter < RP;

  if (t == 0) {
    tc::mbar_init(done, 1);
    tc::fence_barrier_init();
    *bad = 0;
  }
  if (warp == 0) {
    tc::tmem_alloc(tmem_slot, 512);
    tc::tmem_relinquish();
  }

  // U into the places of X (bit for bit), its sum of squares, and the momentum on the way.  A task is
  // 8 neighbours in memory: 8 columns of a row of X, or 8 rows of a column of the transposed one.
  const int tn = mi / s.groups;
  const size_t base = (size_t)(mi % s.groups) * s.rows * s.cols;
  const int tasks = mine * 8 * RP;
  struct Task {
    int r, l, here;   // first element, how many of the 8 are the matrix's
    size_t at;        // in the tensor's matrix
    uint32_t off;     // of the first element in a plane of X
  };
  auto task_of = [&](int k) {
    Task x;
    if (s.tr) {
      x.r = k % (RP / 8) * 8;
      x.l = c_lo * 64 + k / (RP / 8);
      x.here = x.l < s.L ? max(0, min(8, s.R - x.r)) : 0;
      x.at = (size_t)x.l * s.cols + x.r;
    } else {
      x.r = k / (mine * 8);
      x.l = c_lo * 64 + k % (mine * 8) * 8;
      x.here = x.r < s.R ? max(0, min(8, s.L - x.l)) : 0;
      x.at = (size_t)x.r * s.cols + x.l;
    }
    x.off = (uint32_t)(x.l / 64 - c_lo) * kChunk + sw128(x.r, x.l % 64 * 2);
    return x;
  };
  // rows r .. r + 7 of a column start on a swizzle period: row r + i is at i * 128 with the 16-byte
  // block i of the row exchanged
  auto down = [&](const Task& x, int i) { return (x.off + 128u * i) ^ ((uint32_t)i << 4); };
  auto put8 = [&](const Task& x, uint4 hi, uint4 lo) {
    if (!s.tr) {
      *reinterpret_cast<uint4*>(xh + x.off) = hi;
      *reinterpret_cast<uint4*>(xl + x.off) = lo;
    } else {
      const uint16_t *h = reinterpret_cast<const uint16_t*>(&hi), *l = reinterpret_cast<const uint16_t*>(&lo);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        *reinterpret_cast<uint16_t*>(xh + down(x, i)) = h[i];
        *reinterpret_cast<uint16_t*>(xl + down(x, i)) = l[i];
      }
    }
  };
  auto get8 = [&](const Task& x, uint4& hi, uint4& lo) {
    if (!s.tr) {
      hi = *reinterpret_cast<const uint4*>(xh + x.off);
      lo = *reinterpret_cast<const uint4*>(xl + x.off);
    } else {
      alignas(16) uint16_t h[8], l[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        h[i] = *reinterpret_cast<const uint16_t*>(xh + down(x, i));
        l[i] = *reinterpret_cast<const uint16_t*>(xl + down(x, i));
      }
      hi = *reinterpret_cast<const uint4*>(h);
      lo = *reinterpret_cast<const uint4*>(l);
    }
  };
  {
    const T* in = static_cast<const T*>(ptr.in[tn]) + base;
    const float* m = a.r.step ? ptr.m[tn] + base : nullptr;
    float* mo = a.r.step ? ptr.m_out[tn] + base : nullptr;
    double sum = 0.0;
#pragma unroll 2
    for (int k = t; k < tasks; k += kSmallThreads) {
      const Task x = task_of(k);
      float u[8] = {};
      if (x.here > 0) {
        load_wide(in + x.at, x.here, u);
        if (a.r.step) {
          float v[8];
          load_wide(m + x.at, x.here, v);
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] = new_momentum(a.r, u[i], v[i]);
          store_wide(mo + x.at, x.here, v);
#pragma unroll
          for (int i = 0; i < 8; ++i) u[i] = i < x.here ? update_of(a.r, u[i], v[i]) : 0.0f;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) sum = fma((double)u[i], (double)u[i], sum);
      }
      uint4 hi, lo;
      bits8(u, hi, lo);
      put8(x, hi, lo);
    }
    sum = warp_sum(sum);
    if (lane == 0) warps[warp] = sum;
  }
  tc::fence_before_sync();
  if (S > 1) cluster_sync();  // everyone's shared memory may be written from here on
  else __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  if (t < S) {
    double v = 0.0;
    for (int k = 0; k < kSmallThreads / 32; ++k) v += warps[k];
    if (S > 1) st_remote(at_rank(tc::smem_u32(&norms[q]), t), v);
    else norms[0] = v;
  }
  if (S > 1) cluster_sync();
  else __syncthreads();
  double all = 0.0;
  for (int k = 0; k < S; ++k) all += norms[k];
  const float scale = (float)((double)kSx / (sqrt(all) + a.eps));
  for (int k = t; k < tasks; k += kSmallThreads) {
    const Task x = task_of(k);
    uint4 hi, lo;
    float v[8];
    get8(x, hi, lo);
    unbits8(hi, lo, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] *= scale;
    split8(v, hi, lo);
    put8(x, hi, lo);
  }
  tc::fence_proxy_async();
  __syncthreads();

  uint32_t phase = 0;
  bool ok = true;
  const unsigned long long limit = a.hold_ns ? a.hold_ns : tc::kWaitNs;
  const uint32_t sxh = tc::smem_u32(xh), sxl = tc::smem_u32(xl), sah = tc::smem_u32(ah), sal = tc::smem_u32(al);
  const uint32_t tw = tmem + ((uint32_t)quarter << 16);
  auto finish = [&]() {  // the issued products are done and visible; a warp waits in vain once
    ok = ok && __all_sync(~0u, tc::mbar_wait(done, phase, limit));
    phase ^= 1;
    tc::fence_after_sync();
  };
  auto settle = [&]() {  // shared memory as written by all, TMEM as read by all, before the next products
    tc::fence_proxy_async();
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
  };
  // P P^T of hi and lo planes with K-major chunks, K = 64 * chunks.  The large products of the chunks
  // go round kSums accumulators, which keeps the chains short that the tensor core cuts.
  constexpr int kSums = RP == 64 ? 4 : 3;
  auto sum_at = [](int j) -> uint32_t { return RP == 64 ? 256 + 64 * j : j < 2 ? 256 + 128 * j : 0; };
  auto square = [&](uint32_t ph, uint32_t pl, int chunks) {
    constexpr uint32_t idesc = idesc_f16(128, RP, false, false);
    for (int k = 0; k < 4 * chunks; ++k) {
      const uint32_t off = (uint32_t)(k >> 2) * kChunk + (k & 3) * 32;
      const uint64_t h = tc::desc_sw128(ph + off, 16, 1024);
      tc::mma_bf16(tmem + sum_at((k >> 2) % kSums), h, h, idesc, k >= 4 * kSums || (k & 3) != 0);
      const uint64_t l = tc::desc_sw128(pl + off, 16, 1024);
      tc::mma_bf16(tmem + 128, h, l, idesc, k != 0);
      tc::mma_bf16(tmem + 128, l, h, idesc, 1);
    }
    tc::mma_commit(done);
  };
  // 16 columns of a lane's row of that product
  auto drain = [&](int c, int chunks, float (&v)[16]) {
    uint32_t e[16];
    tc::tmem_ld16(tw + sum_at(0) + c, v);
#pragma unroll
    for (int j = 1; j < kSums; ++j) {
      if (j < chunks) {
        tc::tmem_ld_chunks<1>(tw + sum_at(j) + c, e);
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] += __uint_as_float(e[i]);
      }
    }
    tc::tmem_ld_chunks<1>(tw + 128 + c, e);
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = fmaf(__uint_as_float(e[i]), 1.0f / kSl, v[i]);
  };
  constexpr int kRun = RP / kSides;  // columns of A a warp drains
  constexpr float kToA = kSa / (kSx * kSx);
  const int shift = 31 - __clz(RP / S);  // log2 of a block of A's columns
  for (int step = 0; step < a.steps; ++step) {
    if (t == 0 && ok && !(a.hold_ns && step == 0 && q == 0)) square(sxh, sxl, mine);
    __syncwarp();
    finish();
    if (S > 1) {
      if (live) {
#pragma unroll
        for (int c = side * kRun; c < (side + 1) * kRun; c += 16) {
          float v[16];
          drain(c, mine, v);
#pragma unroll
          for (int h = 0; h < 16; h += 8) {  // a block has 8 columns at least; a warp's row is 128 bytes
            const int col = c + h, dst = col >> shift, at = (q << shift) + (col & ((1 << shift) - 1));
            const uint32_t to = at_rank(tc::smem_u32(recv + at * RP + row), dst);
#pragma unroll
            for (int i = 0; i < 8; ++i) st_remote(to + i * RP * 4, v[h + i]);
          }
        }
      }
      tc::fence_before_sync();
      cluster_sync();
      // rows of block q of A (A is symmetric), 8 columns a task, to every CTA
      for (int task = t; task < (RP / 8) << shift; task += kSmallThreads) {
        const int j = task / (RP / 8), i0 = task % (RP / 8) * 8;
        float v[8] = {};
#pragma unroll 4
        for (int k = 0; k < S; ++k) {
          const float4* p = reinterpret_cast<const float4*>(recv + ((k << shift) + j) * RP + i0);
          const float4 x = p[0], y = p[1];
          v[0] += x.x;
          v[1] += x.y;
          v[2] += x.z;
          v[3] += x.w;
          v[4] += y.x;
          v[5] += y.y;
          v[6] += y.z;
          v[7] += y.w;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] *= kToA;
        uint4 hi, lo;
        split8(v, hi, lo);
        const uint32_t off = (uint32_t)(i0 / 64) * kChunk + sw128((q << shift) + j, i0 % 64 * 2);
        for (int k = 0; k < S; ++k) {
          st_remote(at_rank(sah + off, k), hi);
          st_remote(at_rank(sal + off, k), lo);
        }
      }
      fence_proxy_async_all();
      cluster_sync();
      tc::fence_after_sync();
      fence_proxy_async_all();
    } else {
      if (live) {
#pragma unroll
        for (int c = side * kRun; c < (side + 1) * kRun; c += 16) {
          float v[16];
          drain(c, mine, v);
#pragma unroll
          for (int h = 0; h < 16; h += 8) {
            float w[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i] = v[h + i] * kToA;
            const uint32_t off = (uint32_t)((c + h) / 64) * kChunk + sw128(row, (c + h) % 64 * 2);
            uint4 hi, lo;
            split8(w, hi, lo);
            *reinterpret_cast<uint4*>(ah + off) = hi;
            *reinterpret_cast<uint4*>(al + off) = lo;
          }
        }
      }
      settle();
    }
    if (t == 0 && ok) square(sah, sal, RP / 64);
    __syncwarp();
    finish();
    if (live) {
#pragma unroll
      for (int c = side * kRun; c < (side + 1) * kRun; c += 16) {
        float v[16];
        drain(c, RP / 64, v);
#pragma unroll
        for (int h = 0; h < 16; h += 8) {
          const uint32_t off = (uint32_t)((c + h) / 64) * kChunk + sw128(row, (c + h) % 64 * 2);
          float w[8];
          join8(*reinterpret_cast<const uint4*>(ah + off), *reinterpret_cast<const uint4*>(al + off), w);
#pragma unroll
          for (int i = 0; i < 8; ++i)
            w[i] = fmaf(a.c * (kSb / (kSa * kSa)), v[h + i],
                        fmaf(a.b * (kSb / kSa), w[i], row == c + h + i ? a.a * kSb : 0.0f));
          uint4 hi, lo;
          split8(w, hi, lo);
          *reinterpret_cast<uint4*>(ah + off) = hi;
          *reinterpret_cast<uint4*>(al + off) = lo;
        }
      }
    }
    settle();
    const bool last = step + 1 == a.steps;
    for (int g0 = 0; g0 < mine; g0 += 4) {  // up to 256 columns at a time
      const int cols = min(4, mine - g0) * 64;
      if (t == 0 && ok) {
        const uint32_t idesc = idesc_f16(128, cols, false, true);
        for (int k = 0; k < RP / 16; ++k) {
          const uint32_t poff = (uint32_t)(k >> 2) * kChunk + (k & 3) * 32, qoff = (uint32_t)g0 * kChunk + k * 2048;
          const uint64_t bh = tc::desc_sw128(sah + poff, 16, 1024);
          const uint64_t yh = tc::desc_sw128(sxh + qoff, kChunk, 1024), yl = tc::desc_sw128(sxl + qoff, kChunk, 1024);
          tc::mma_bf16(tmem, bh, yh, idesc, k != 0);
          tc::mma_bf16(tmem + 256, bh, yl, idesc, k != 0);
          tc::mma_bf16(tmem + 256, tc::desc_sw128(sal + poff, 16, 1024), yh, idesc, 1);
        }
        tc::mma_commit(done);
      }
      __syncwarp();
      finish();
      if (last && g0 + 4 >= mine) {  // the last wait
        if (!ok) mark_bad(bad, S);
        if (S > 1) cluster_arrive();
      }
      if (live) {
        for (int c = side * (cols / kSides); c < (side + 1) * (cols / kSides); c += 16) {
          float v[16];
          drain16(tw + c, tw + 256 + c, v);
#pragma unroll
          for (int h = 0; h < 16; h += 8) {
            float w[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i] = v[h + i] * (last ? 1.0f / (kSb * kSx) : 1.0f / kSb);
            uint4 hi, lo;
            if (last) bits8(w, hi, lo);
            else split8(w, hi, lo);
            const uint32_t off = (uint32_t)(g0 + (c + h) / 64) * kChunk + sw128(row, (c + h) % 64 * 2);
            *reinterpret_cast<uint4*>(xh + off) = hi;
            *reinterpret_cast<uint4*>(xl + off) = lo;
          }
        }
      }
      settle();
    }
  }
  if (S > 1) cluster_wait();
  const bool store = *reinterpret_cast<volatile int*>(bad) == 0;
  if (store) {
    T* out = static_cast<T*>(ptr.out[tn]) + base;
    const T* w = a.r.step ? static_cast<const T*>(ptr.w[tn]) + base : nullptr;
#pragma unroll 2
    for (int k = t; k < tasks; k += kSmallThreads) {
      const Task x = task_of(k);
      if (x.here <= 0) continue;
      uint4 hi, lo;
      float v[8];
      get8(x, hi, lo);
      unbits8(hi, lo, v);
      float o[8] = {};
      if (a.r.step) load_wide(w + x.at, x.here, o);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = result_of(a.r, o[i], v[i]);
      store_wide(out + x.at, x.here, v);
    }
  }
  if (!store) tc::give_up();
  if (warp == 0) tc::tmem_dealloc(tmem, 512);
}

// ------------------------------------------------------------------ thin matrices: one launch, fp32
//
// Up to 32 rows are too few for the tensor core, whose M is 128 and whose answers take half a
// microsecond: three waits a step.  Here X stays in shared memory as fp32 columns of RP values, in
// plain fp32 arithmetic.  A cluster of S CTAs takes one matrix, each a run of its columns; only the
// shares of X X^T (RP x RP) cross the cluster, each CTA sends its own to all and adds all in the same
// order.  What bounds it is latency: four barriers a step, and one of the cluster.
//
// X X^T: a thread takes a 4 x 4 block of it over every (512 / blocks)-th column, 16 multiply-adds for
// two 16-byte reads, and the partial blocks are added through shared memory.  B X: a task is one
// column and 8 (or 4) rows of B, the column in registers, B's rows read as broadcasts.

constexpr int kThinThreads = 512;

struct ThinArgs {
  Shape s;
  Rule r;
  float a, b, c;
  double eps;
  int steps, S, most;  // most: columns of a CTA
};

// Floats of a CTA's shared memory: two buffers of X, then A, B and the shares of two steps.
struct ThinLayout {
  int pitch, buffer, a, b, recv, total;
};
__host__ __device__ constexpr ThinLayout thin_layout(int rp, int S, int most) {
  ThinLayout l{};
  l.pitch = rp + 4;  // neighbouring columns lie 4 banks apart
  // the idle buffer also holds the partial blocks of X X^T, 16 values a thread
  l.buffer = most * l.pitch > kThinThreads * 16 ? most * l.pitch : kThinThreads * 16;
  l.a = 2 * l.buffer;
  l.b = l.a + rp * rp;
  l.recv = l.b + rp * rp;
  l.total = l.recv + (S > 1 ? 2 * S * rp * rp : 0);
  return l;
}

template <typename T, int RP>
__global__ void __launch_bounds__(kThinThreads, 1)
    ns_thin_kernel(const __grid_constant__ Pointers ptr, const __grid_constant__ ThinArgs g) {
  extern __shared__ __align__(16) float thin[];
  __shared__ double norms[kSmallMaxCluster], warps[kThinThreads / 32];
  constexpr int E = RP * RP, kBlocks = (RP / 4) * (RP / 4), kParts = kThinThreads / kBlocks;
  const ThinLayout lay = thin_layout(RP, g.S, g.most);
  const Shape& s = g.s;
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const int S = g.S, q = S > 1 ? (int)cluster_rank() : 0, mi = blockIdx.x / S;
  const int l_lo = (int)((long long)s.L * q / S), mine = (int)((long long)s.L * (q + 1) / S) - l_lo;
  const int tn = mi / s.groups;
  const size_t base = (size_t)(mi % s.groups) * s.rows * s.cols;
  float* now = thin;
  float* next = thin + lay.buffer;
  float *am = thin + lay.a, *bm = thin + lay.b;
  // element k of this CTA's columns, neighbours in k neighbours in memory
  const int total = s.R * mine;
  auto place = [&](int k, int& at, size_t& gl) {
    int r, l;
    if (s.tr) {
      l = k / s.R;
      r = k - l * s.R;
      gl = (size_t)(l_lo + l) * s.cols + r;
    } else {
      r = k / mine;
      l = k - r * mine;
      gl = (size_t)r * s.cols + l_lo + l;
    }
    at = l * lay.pitch + r;
  };
  for (int k = t; k < mine * lay.pitch; k += kThinThreads) now[k] = 0.0f;  // rows R.. of a column
  __syncthreads();
  {
    const T* in = static_cast<const T*>(ptr.in[tn]) + base;
    const float* m = g.r.step ? ptr.m[tn] + base : nullptr;
    float* mo = g.r.step ? ptr.m_out[tn] + base : nullptr;
    double sum = 0.0;
#pragma unroll 4
    for (int k = t; k < total; k += kThinThreads) {
      int at;
      size_t gl;
      place(k, at, gl);
      float u = to_f32(in[gl]);
      if (g.r.step) {
        const float v = new_momentum(g.r, u, m[gl]);
        mo[gl] = v;
        u = update_of(g.r, u, v);
      }
      now[at] = u;
      sum = fma((double)u, (double)u, sum);
    }
    sum = warp_sum(sum);
    if (lane == 0) warps[warp] = sum;
  }
  if (S > 1) cluster_sync();  // everyone's shared memory may be written from here on
  else __syncthreads();
  if (t < S) {
    double v = 0.0;
    for (int k = 0; k < kThinThreads / 32; ++k) v += warps[k];
    if (S > 1) st_remote(at_rank(tc::smem_u32(&norms[q]), t), v);
    else norms[0] = v;
  }
  if (S > 1) cluster_sync();
  else __syncthreads();
  double all = 0.0;
  for (int k = 0; k < S; ++k) all += norms[k];
  const float scale = (float)(1.0 / (sqrt(all) + g.eps));
  for (int k = t; k < mine * lay.pitch; k += kThinThreads) now[k] *= scale;
  __syncthreads();

  for (int step = 0; step < g.steps; ++step) {
    {  // partial blocks of X X^T into the idle buffer: [part][block][16]
      const int blk = t % kBlocks, bi = blk / (RP / 4) * 4, bj = blk % (RP / 4) * 4;
      float acc[16] = {};
#pragma unroll 2
      for (int l = t / kBlocks; l < mine; l += kParts) {
        const float4 x = *reinterpret_cast<const float4*>(now + l * lay.pitch + bi);
        const float4 y = *reinterpret_cast<const float4*>(now + l * lay.pitch + bj);
        const float xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[4 * i + j] = fmaf(xs[i], ys[j], acc[4 * i + j]);
      }
      // value e of a thread at e * 512 + t: no bank conflicts
#pragma unroll
      for (int e = 0; e < 16; ++e) next[e * kThinThreads + t] = acc[e];
    }
    __syncthreads();
    float* recv = thin + lay.recv + (step & 1) * S * E;
    {  // entry e: its kParts values, by kLanes lanes
      constexpr int kLanes = E < kThinThreads ? kThinThreads / E : 1;
#pragma unroll
      for (int e = t / kLanes; e < E; e += kThinThreads / kLanes) {
        const int i = e / RP, j = e % RP, blk = i / 4 * (RP / 4) + j / 4, v = i % 4 * 4 + j % 4;
        float sum = 0.0f;
#pragma unroll 4
        for (int p = t % kLanes; p < kParts; p += kLanes) sum += next[v * kThinThreads + p * kBlocks + blk];
#pragma unroll
        for (int m = 1; m < kLanes; m <<= 1) sum += __shfl_xor_sync(~0u, sum, m);
        if (t % kLanes == 0) {
          if (S > 1) {
            for (int k = 0; k < S; ++k) st_remote(at_rank(tc::smem_u32(recv + q * E + e), k), sum);
          } else {
            am[e] = sum;
          }
        }
      }
    }
    if (S > 1) {
      cluster_sync();
      for (int e = t; e < E; e += kThinThreads) {
        float sum = 0.0f;
        for (int k = 0; k < S; ++k) sum += recv[k * E + e];
        am[e] = sum;
      }
    }
    __syncthreads();
    if (t < E) {  // entries of one column of A A, rows 512 / RP apart
      constexpr int kPer = E > kThinThreads ? E / kThinThreads : 1, kApart = kThinThreads / RP;
      const int i = t / RP, j = t % RP;
      float sum[kPer] = {};
#pragma unroll
      for (int k = 0; k < RP; k += 4) {
        const float c[4] = {am[k * RP + j], am[(k + 1) * RP + j], am[(k + 2) * RP + j], am[(k + 3) * RP + j]};
#pragma unroll
        for (int p = 0; p < kPer; ++p) {
          const float4 r = *reinterpret_cast<const float4*>(am + (i + p * kApart) * RP + k);
          sum[p] = fmaf(r.x, c[0], sum[p]);
          sum[p] = fmaf(r.y, c[1], sum[p]);
          sum[p] = fmaf(r.z, c[2], sum[p]);
          sum[p] = fmaf(r.w, c[3], sum[p]);
        }
      }
#pragma unroll
      for (int p = 0; p < kPer; ++p) {
        const int row = i + p * kApart, e = row * RP + j;
        bm[e] = fmaf(g.c, sum[p], fmaf(g.b, am[e], row == j ? g.a : 0.0f));
      }
    }
    __syncthreads();
    {
      constexpr int kTake = RP < 8 ? RP : 8, kSets = RP / kTake;
      const int tasks = mine * kSets;
      for (int k = t; k < tasks; k += kThinThreads) {
        const int set = kSets == 1 ? 0 : k / mine, l = kSets == 1 ? k : k - set * mine;
        float x[RP];
#pragma unroll
        for (int i = 0; i < RP; i += 4) {
          const float4 v = *reinterpret_cast<const float4*>(now + l * lay.pitch + i);
          x[i] = v.x;
          x[i + 1] = v.y;
          x[i + 2] = v.z;
          x[i + 3] = v.w;
        }
#pragma unroll
        for (int h = 0; h < kTake; h += 4) {
          float o[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float4* b = reinterpret_cast<const float4*>(bm + (set * kTake + h + i) * RP);
            float sum = 0.0f;
#pragma unroll
            for (int j = 0; j < RP; j += 4) {
              const float4 v = b[j / 4];
              sum = fmaf(v.x, x[j], sum);
              sum = fmaf(v.y, x[j + 1], sum);
              sum = fmaf(v.z, x[j + 2], sum);
              sum = fmaf(v.w, x[j + 3], sum);
            }
            o[i] = sum;
          }
          *reinterpret_cast<float4*>(next + l * lay.pitch + set * kTake + h) = make_float4(o[0], o[1], o[2], o[3]);
        }
      }
    }
    __syncthreads();
    float* swap = now;
    now = next;
    next = swap;
  }
  T* out = static_cast<T*>(ptr.out[tn]) + base;
  const T* w = g.r.step ? static_cast<const T*>(ptr.w[tn]) + base : nullptr;
#pragma unroll 4
  for (int k = t; k < total; k += kThinThreads) {
    int at;
    size_t gl;
    place(k, at, gl);
    out[gl] = from_f32<T>(result_of(g.r, g.r.step ? to_f32(w[gl]) : 0.0f, now[at]));
  }
}

// ------------------------------------------------------------------ host side

int up(int v, int to) { return (v + to - 1) / to * to; }

Shape shape_of(int n, int groups, int rows, int cols) {
  Shape s{};
  s.groups = groups;
  s.rows = rows;
  s.cols = cols;
  s.tr = rows > cols;
  s.R = std::min(rows, cols);
  s.L = std::max(rows, cols);
  s.nm = n * groups;
  // pairs of CTAs where there is a tile for nearly every one of them and more than one along R
  // (1024 x 4608: 341 us on pairs, 427 on single CTAs; 24 of 256 x 768: 215 and 201)
  s.tile = s.R > 256 && (long long)s.nm * up(s.R, 256) * up(s.L, 256) / (256 * 256) >= 64 ? 256 : 128;
  s.Rp = up(s.R, s.tile);
  s.Lp = up(s.L, s.tile);
  return s;
}

// Parts of the K range of a product.
// Pairs (symmetric products only): as many as give every two SMs a pair, each of 256 values at least,
// unless the second kernel that they need (7 us) costs more than the chunks (1 us) that they save.
// Single CTAs: a cluster as large as there are SMs for all tiles', for 512 values at least (a chunk takes
// 0.75 us, the exchange 3 us; 300 x 513 in 147 us, without clusters 157, and from 256 values on 142 with 12 of
// 200 x 300 in 126 either way).  148 SMs run some 16 clusters of 8, 32 of 4 and 70 of 2 at a time, and other
// devices their share of that.
int splits_of(const Shape& s, long long tiles, int k, int sms) {
  const int chunks = k / kBk;
  if (s.tile == 256) {
    const int S = std::max(1, std::min({(int)std::max<long long>(1, sms / 2 / tiles), chunks / 4, kMaxSplits}));
    return chunks - chunks / S < 7 ? 1 : S;
  }
  return chunks < kLeastJoin ? 1 : 9 * tiles <= sms ? 8 : 9 * tiles <= 2 * sms ? 4 : 19 * tiles <= 9 * sms ? 2 : 1;
}
long long symmetric_tiles(const Shape& s) {
  const long long nt = s.Rp / s.tile;
  return nt * (nt + 1) / 2 * s.nm;
}

// The next kernel of a chain, brought up while the one before it runs.
template <typename K, typename... A>
cudaError_t chain(K k, dim3 grid, int cluster, int threads, size_t smem, cudaStream_t st, A... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, k, args...);
  count_launch();
  return e != cudaSuccess ? e : cudaGetLastError();
}

size_t align256(size_t v) { return (v + 255) & ~size_t(255); }

constexpr int kMostSms = 160;  // what the workspace provides for

struct Layout {
  size_t x[2], a, b, part, norm, fail, total;
};

Layout layout_of(const Shape& s) {
  Layout l{};
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t r = at;
    at += align256(bytes);
    return r;
  };
  const size_t nx = (size_t)s.nm * s.Rp * s.Lp, na = (size_t)s.nm * s.Rp * s.Rp;
  l.x[0] = take(4 * nx);
  l.x[1] = take(4 * nx);
  l.a = take(4 * na);
  l.b = take(4 * na);
  if (s.tile == 256) {
    const long long t = symmetric_tiles(s);
    l.part = take(4 * na * std::max(splits_of(s, t, s.Lp, kMostSms), splits_of(s, t, s.Rp, kMostSms)));
  }
  l.norm = take(sizeof(double) * s.nm * kNormBlocks);
  l.fail = take(sizeof(int));
  l.total = at;
  return l;
}

// fp16 map of [z][rows][cols] with boxes of 64 x 64.
bool plane_map(CUtensorMap* m, const void* base, int cols, int rows, int z) {
  tc::EncodeTiledFn f = tc::encode_tiled_fn();
  if (!f) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, (cuuint64_t)z};
  const cuuint64_t strides[2] = {(cuuint64_t)cols * 2, (cuuint64_t)cols * rows * 2};
  const cuuint32_t box[3] = {64, 64, 1}, es[3] = {1, 1, 1};
  return f(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<void*>(base), dims, strides, box, es,
           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

constexpr size_t kProductSmem = kStages * kStageBytes + 1024 + 128;

template <typename T, Product MODE, Team TEAM>
cudaError_t product_by(const CUtensorMap& p, const CUtensorMap& q, const Pointers& ptr, const ProductArgs& a,
                       cudaStream_t st) {
  auto k = ns_product_kernel<T, MODE, TEAM>;
  cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kProductSmem);
  if (e != cudaSuccess) return e;
  const int tiles = MODE == kSymmetric ? a.tn * (a.tn + 1) / 2 : a.tm * a.tn, ctas = TEAM == kPair ? 2 : 1;
  return chain(k, dim3(ctas * tiles * a.S, a.s.nm), TEAM == kPair ? 2 : TEAM == kJoined ? a.S : 1, kProductThreads,
               kProductSmem, st, p, q, ptr, a);
}

template <typename T, Product MODE>
cudaError_t product(const CUtensorMap& p, const CUtensorMap& q, const Pointers& ptr, const ProductArgs& a,
                    cudaStream_t st) {
  if (a.s.tile == 256) return product_by<T, MODE, kPair>(p, q, ptr, a, st);
  return a.S > 1 ? product_by<T, MODE, kJoined>(p, q, ptr, a, st) : product_by<T, MODE, kAlone>(p, q, ptr, a, st);
}

struct SmallPlan {
  bool ok = false;
  int S = 0, nc = 0, max_chunks = 0, rp = 0;
  size_t smem = 0;
};

// The one-launch form serves up to 128 rows whose columns fit the shared memory of a cluster.  A
// step costs as much as three chunks besides its CTA's own, and the exchange between CTAs one more
// (measured: 48 matrices of 64 x 576 in 77, 58 and 85 us on clusters of 1, 2 and 4).
SmallPlan small_plan(const Shape& s, int sms) {
  SmallPlan p;
  if (s.R > 128) return p;
  p.rp = s.R <= 64 ? 64 : 128;
  p.nc = (s.L + 63) / 64;
  long long best = 0;
  for (int S = 1; S <= kSmallMaxCluster && S <= p.nc; S *= 2) {
    const int most = (p.nc + S - 1) / S;
    const size_t smem = small_layout(p.rp, S, most).total + 1024;
    if (smem > kSmallSmem) continue;
    const long long waves = ((long long)s.nm * S + sms - 1) / sms, cost = waves * (most + 3 + (S > 1 ? 1 : 0));
    if (p.ok && cost >= best) continue;
    best = cost;
    p.ok = true;
    p.S = S;
    p.max_chunks = most;
    p.smem = std::max(smem, kSmallLeast);
  }
  return p;
}

template <typename K, typename... A>
cudaError_t launch_clusters(K k, int ctas, int cluster, int threads, size_t smem, cudaStream_t st, const A&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)ctas);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)cluster;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, k, args...);
  count_launch();
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <typename T, int RP>
cudaError_t run_small(const Pointers& ptr, const SmallArgs& a, size_t smem, cudaStream_t st) {
  auto k = ns_small_kernel<T, RP>;
  // the same limit in every call: another thread may be between its own two calls here
  cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmallSmem);
  if (e != cudaSuccess) return e;
  return launch_clusters(k, a.s.nm * a.S, a.S, kSmallThreads, smem, st, ptr, a);
}

struct ThinPlan {
  bool ok = false;
  int S = 0, most = 0, rp = 0;
  size_t smem = 0;
};

// Up to 32 rows: the smallest cluster whose CTAs have little enough to do (24 columns of 32 rows or as
// much work of fewer: 32 x 96 takes 22 us on one CTA and 18.2 on four, 9 x 2000 takes 50 on one, 43 on
// two and 21 on eight) and fit shared memory, as far as there are SMs for all matrices.
ThinPlan thin_plan(const Shape& s, int sms) {
  ThinPlan p;
  if (s.R > 32) return p;
  p.rp = s.R <= 4 ? 4 : s.R <= 8 ? 8 : s.R <= 16 ? 16 : 32;
  for (int S = 1; S <= kSmallMaxCluster && S <= s.L; S *= 2) {
    const int most = (s.L + S - 1) / S;
    const size_t smem = (size_t)thin_layout(p.rp, S, most).total * sizeof(float);
    if (smem > kSmallSmem) continue;
    if (p.ok && (long long)s.nm * S > sms) break;
    p.ok = true;
    p.S = S;
    p.most = most;
    p.smem = smem;
    if ((long long)most * p.rp * p.rp <= 24 * 1024) break;
  }
  return p;
}

template <typename T, int RP>
cudaError_t run_thin(const Pointers& ptr, const ThinArgs& a, size_t smem, cudaStream_t st) {
  auto k = ns_thin_kernel<T, RP>;
  cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmallSmem);
  return e != cudaSuccess ? e : launch_clusters(k, a.s.nm * a.S, a.S, kThinThreads, smem, st, ptr, a);
}

cudaError_t sm_count(int* sms) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  return e != cudaSuccess ? e : cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev);
}

template <typename T>
cudaError_t run_chunk(const MuonArgs& a, int t0, int n, char* ws, int sms, cudaStream_t st) {
  const Shape s = shape_of(n, a.groups, a.rows, a.cols);
  const Layout l = layout_of(s);
  Pointers ptr{};
  for (int i = 0; i < n; ++i) {
    ptr.in[i] = a.in[t0 + i];
    ptr.out[i] = a.out[t0 + i];
    if (a.step) {
      ptr.w[i] = a.w[t0 + i];
      ptr.m[i] = a.m[t0 + i];
      ptr.m_out[i] = a.m_out[t0 + i];
    }
  }
  Rule r{a.step, a.nesterov, a.momentum, a.keep, a.rate};
  const ThinPlan tp = thin_plan(s, sms);
  if (tp.ok) {
    const ThinArgs g{s, r, a.a, a.b, a.c, a.eps, a.steps, tp.S, tp.most};
    switch (tp.rp) {
      case 4: return run_thin<T, 4>(ptr, g, tp.smem, st);
      case 8: return run_thin<T, 8>(ptr, g, tp.smem, st);
      case 16: return run_thin<T, 16>(ptr, g, tp.smem, st);
      default: return run_thin<T, 32>(ptr, g, tp.smem, st);
    }
  }
  const SmallPlan sp = small_plan(s, sms);
  if (sp.ok) {
    const SmallArgs g{s, r, a.a, a.b, a.c, a.eps, a.steps, sp.S, sp.nc, sp.max_chunks, a.hold_ns};
    return sp.rp == 64 ? run_small<T, 64>(ptr, g, sp.smem, st) : run_small<T, 128>(ptr, g, sp.smem, st);
  }
  __half* x[2] = {reinterpret_cast<__half*>(ws + l.x[0]), reinterpret_cast<__half*>(ws + l.x[1])};
  __half* am = reinterpret_cast<__half*>(ws + l.a);
  __half* bm = reinterpret_cast<__half*>(ws + l.b);
  float* part = reinterpret_cast<float*>(ws + l.part);
  double* norm = reinterpret_cast<double*>(ws + l.norm);
  int* fail = reinterpret_cast<int*>(ws + l.fail);
  CUtensorMap mx[2], ma, mb;
  if (!plane_map(&mx[0], x[0], s.Lp, s.Rp, 2 * s.nm) || !plane_map(&mx[1], x[1], s.Lp, s.Rp, 2 * s.nm) ||
      !plane_map(&ma, am, s.Rp, s.Rp, 2 * s.nm) || !plane_map(&mb, bm, s.Rp, s.Rp, 2 * s.nm))
    return cudaErrorInvalidValue;
  cudaError_t e;
  const int blocks = (int)std::min<size_t>(kNormBlocks, ((size_t)a.rows * a.cols + 256 * kWide - 1) / (256 * kWide));
  ns_norm_kernel<T><<<dim3(blocks, s.nm), 256, 0, st>>>(ptr, s, r, norm, fail);
  count_launch();
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  if ((e = chain(ns_load_kernel<T>, dim3(s.Lp / 64, s.Rp / 64, s.nm), 1, 256, 0, st, ptr, s, r, a.eps,
                 (const double*)norm, blocks, x[0])) != cudaSuccess)
    return e;
  ProductArgs g{};
  g.s = s;
  g.r = r;
  g.part = part;
  g.fail = fail;
  const dim3 red(s.Rp / 64, s.Rp / 64, s.nm);
  // P P^T into dst, as `f` says
  auto square = [&](const CUtensorMap& p, int k, const Becomes& f, __half* dst) {
    g.upper = f.am != nullptr;
    g.tm = g.tn = s.Rp / s.tile;
    g.chunks = k / kBk;
    g.S = splits_of(s, symmetric_tiles(s), k, sms);
    g.f = f;
    g.dst = dst;
    cudaError_t err = product<T, kSymmetric>(p, p, ptr, g, st);
    if (err == cudaSuccess && s.tile == 256 && g.S > 1) err = chain(ns_reduce_kernel, red, 1, 256, 0, st, (const float*)part, s, g.S, f, dst);
    return err;
  };
  for (int k = 0; k < a.steps; ++k) {
    const int now = k & 1;
    g.hold_ns = k == 0 ? a.hold_ns : 0;
    if ((e = square(mx[now], s.Lp, Becomes{a.a, a.b, a.c, nullptr}, am)) != cudaSuccess) return e;
    g.hold_ns = 0;
    if ((e = square(ma, s.Rp, Becomes{a.a, a.b, a.c, am}, bm)) != cudaSuccess) return e;
    g.upper = true;
    g.chunks = s.Rp / kBk;
    g.tn = s.Lp / s.tile;
    g.S = s.tile == 256 ? 1 : splits_of(s, (long long)g.tm * g.tn * s.nm, s.Rp, sms);
    g.dst = x[now ^ 1];
    e = k + 1 < a.steps ? product<T, kUpdate>(mb, mx[now], ptr, g, st) : product<T, kFinal>(mb, mx[now], ptr, g, st);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace

size_t muon_workspace(int n, int groups, int rows, int cols) {
  const Shape s = shape_of(std::min(n, kTensors), groups, rows, cols);
  if (thin_plan(s, kMostSms).ok || small_plan(s, kMostSms).ok) return 0;
  // the last tensors of many: fewer matrices, but perhaps more parts of K each
  const int rest = n > kTensors ? n % kTensors : 0;
  return std::max(layout_of(s).total, rest ? layout_of(shape_of(rest, groups, rows, cols)).total : 0);
}

cudaError_t launch_muon(const MuonArgs& a, void* workspace, cudaStream_t st) {
  int sms = 0;
  cudaError_t q = sm_count(&sms);
  if (q != cudaSuccess) return q;
  sms = std::min(sms, kMostSms);
  for (int t0 = 0; t0 < a.n; t0 += kTensors) {
    const int n = std::min(kTensors, a.n - t0);
    char* ws = static_cast<char*>(workspace);
    cudaError_t e = a.bf16 ? run_chunk<__nv_bfloat16>(a, t0, n, ws, sms, st) : run_chunk<float>(a, t0, n, ws, sms, st);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

int take_muon_status() {
  int v = 0, z = 0;
  cudaMemcpyFromSymbol(&v, g_device_status, sizeof(int));
  if (v) cudaMemcpyToSymbol(g_device_status, &z, sizeof(int));
  return v;
}

}  // namespace disco
