// A whole mixture-of-experts layer for a few tokens, with FP8 block-scaled experts:
//
//   scores = x router^T;  the k best experts of each token, weights w from softmax or sigmoid
//   y[t] = sum over its experts e of w_e * W2_e (silu(W1_e x) * (W3_e x)),  W13 = [W1; W3]
//
// With few tokens the layer is the stream of the picked experts' weights: 3 D F bytes for
// each of them, everything else is small.  So every weight byte is read from memory once, through
// a ring in shared memory that belongs to the warp that multiplies it (a warp's 16-byte copies
// cover eight rows of 64 bytes), and up to 16 tokens of an expert share it; further tokens of the
// expert read it from L2 again.  The products run on the warp-level tensor instruction (m16n8k16,
// FP16 operands, FP32 sums): at up to 16 tokens per expert it needs about a third of its rate,
// where a tcgen05 tile of 128 rows would need a layout of its own in shared memory, and a block's
// scales applied behind it.  E4M3 values are exact in FP16.  The activations are not quantised: a
// token's row is scaled by a power of two into FP16's range, which is exact for BF16 values down to
// 2^-29 of the row's largest.  The hidden row keeps FP16's 11 bits, since the instruction takes
// both operands in one type: that adds about 1% to the error of a BF16 output.
//
// Within a block of 128 along K the order of the terms is free, so lane t of a quad takes 16
// consecutive elements of a 64-element run for both operands and no data is exchanged.
//
// Four kernels on one stream, each launched while the one before it ends:
//   route    scores in FP32 with compensated sums, top-k, the token rows in FP16
//   product  (up) per 16 tokens of an expert and 16 hidden columns: the gate and up rows over the
//            whole of D; h in FP16 with an exponent per 8 columns, and the row's maximum
//   product  (down) per 16 tokens of an expert and 32 output rows: each (token, expert) pair's
//            share of y in FP32
//   combine  the shares of a token added in the order its experts were picked
// Nothing is added by atomics but a maximum, so the result does not depend on timing.
#include <algorithm>
#include <cstdint>
#include <mutex>
#include <type_traits>

#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math_constants.h>

#include "../../include/biloco.h"
#include "fp8_dev.cuh"
#include "fp8_moe.h"
#include "fp8_ops.h"
#include "internal.h"
#include "ptx.cuh"

namespace biloco {

namespace {

constexpr int kThreads = 256, kWarps = 8;
constexpr int kTiles = 4;                 // 8-row weight tiles of one item
constexpr int kRouteCtas = 8;             // cluster of the route kernel

__device__ __forceinline__ uint32_t mapa_u32(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ uint32_t cta_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}

__device__ __forceinline__ uint32_t f16x2_from_f32(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// Two E4M3 codes -> two FP16 values (exact).
__device__ __forceinline__ uint32_t f16x2_from_e4m3x2(uint32_t codes) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(codes)));
  return r;
}

// 2^e for e in the normal range.
__device__ __forceinline__ float pow2(int e) { return __int_as_float((e + 127) << 23); }

// Exponent e with 2^e <= |largest| < 2^(e+1), from the FP32 bits of a maximum; kept where
// 2^(1 - e), 2^(14 - e) and 2^(e - 14) are normal numbers (2^-127 is not).
__device__ __forceinline__ int exponent_of(uint32_t bits) {
  return min(max(static_cast<int>(bits >> 23) - 127, -100), 127);
}

// ------------------------------------------------------------------ route

// Eight router values as they lie in memory.
template <bool kF32>
struct RouterPiece {
  uint4 q[kF32 ? 2 : 1];
  __device__ __forceinline__ void load(const void* p, long long at, bool in) {
    const uint4* s = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(p) + at * (kF32 ? 4 : 2));
    q[0] = in ? __ldg(s) : make_uint4(0, 0, 0, 0);
    if (kF32) q[kF32] = in ? __ldg(s + 1) : make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ float lo(int i) const {          // value 2 i
    if (kF32) return __uint_as_float((i & 1) ? q[kF32 ? i >> 1 : 0].z : q[kF32 ? i >> 1 : 0].x);
    return bf16_lo(i == 0 ? q[0].x : i == 1 ? q[0].y : i == 2 ? q[0].z : q[0].w);
  }
  __device__ __forceinline__ float hi(int i) const {          // value 2 i + 1
    if (kF32) return __uint_as_float((i & 1) ? q[kF32 ? i >> 1 : 0].w : q[kF32 ? i >> 1 : 0].y);
    return bf16_hi(i == 0 ? q[0].x : i == 1 ? q[0].y : i == 2 ? q[0].z : q[0].w);
  }
};

// Order-preserving integer key of a score: larger is better, 0 stands for "taken".  A score
// that is no number gets 1, below every number; -0 counts as 0.
__device__ __forceinline__ unsigned long long order_key(double v) {
  if (isnan(v)) return 1;
  const unsigned long long b = static_cast<unsigned long long>(__double_as_longlong(v + 0.0));
  return (b >> 63) ? ~b : b | 0x8000000000000000ull;
}

// A cluster of eight CTAs serves kTok tokens: each CTA scores an eighth of the experts for
// all of them (the router is read once per cluster), the first one picks.  Loops are kept
// rolled: one launch of a few CTAs pays for every instruction line it fetches (with the
// selection unrolled over 512 experts the kernel took 18 us, mostly instruction misses).
template <int kTok, bool kF32>
__global__ void __launch_bounds__(kThreads, 1)
moe_route_kernel(const __grid_constant__ MoeArgs a) {
  extern __shared__ __align__(16) uint8_t rows[];                       // [kTok][D] bf16
  __shared__ double score[kTok][kMoeMaxExperts];                        // the scores, then the weights
  __shared__ unsigned long long key[kTok][kMoeMaxExperts];
  __shared__ uint32_t part[kTok][kWarps];
  griddep_launch_dependents();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = static_cast<int>(cta_rank());
  const int t0 = static_cast<int>(blockIdx.x) / kRouteCtas * kTok;
  const int D = a.D, nvec = D / 8, ntok = min(kTok, a.T - t0);
  // the router does not depend on the kernel before this one: the first loads of this warp's
  // first expert are under way while that one ends
  constexpr int kAhead = kF32 ? 5 : 10;               // pieces of 256 columns a lane has in flight
  RouterPiece<kF32> w[kAhead];
  auto load_pieces = [&](int e, int c0) {
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
      w[u].load(a.router, static_cast<long long>(e) * D + (c0 + 32 * u) * 8, e < a.E && c0 + 32 * u < nvec);
  };
  load_pieces(rank + kRouteCtas * warp, lane);
  griddep_wait();
  uint4* const xs = reinterpret_cast<uint4*>(rows);

  // the token rows into shared memory, and each row's largest magnitude
#pragma unroll
  for (int j = 0; j < kTok; ++j) {
    const uint4* x = reinterpret_cast<const uint4*>(a.x + (t0 + min(j, ntok - 1)) * a.ldx);
    uint32_t top = 0;
#pragma unroll 4
    for (int c = tid; c < nvec; c += kThreads) {
      const uint4 q = x[c];
      xs[j * nvec + c] = q;
      const uint32_t m = __vmaxu2(__vmaxu2(q.x & 0x7FFF7FFFu, q.y & 0x7FFF7FFFu),
                                  __vmaxu2(q.z & 0x7FFF7FFFu, q.w & 0x7FFF7FFFu));
      top = max(top, max(m << 16, m & 0xFFFF0000u));
    }
    top = __reduce_max_sync(0xFFFFFFFFu, top);
    if (lane == 0) part[j][warp] = top;
  }
  cluster_barrier();            // also: the first CTA runs, so its shared memory may be written

  // scores: a warp takes whole experts; sums of eight products, compensated over a lane's
  // eights (Kahan), in FP64 over the lanes
  const uint32_t remote = mapa_u32(smem_u32(&score[0][0]), 0);
#pragma unroll 1
  for (int e = rank + kRouteCtas * warp; e < a.E; e += kRouteCtas * kWarps) {
    float s[kTok], comp[kTok];
#pragma unroll
    for (int j = 0; j < kTok; ++j) s[j] = comp[j] = 0.0f;
#pragma unroll 1
    for (int c0 = lane; c0 < nvec; c0 += 32 * kAhead) {
      if (c0 != lane || e != rank + kRouteCtas * warp) load_pieces(e, c0);
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        if (c0 + 32 * u >= nvec) break;
#pragma unroll
        for (int j = 0; j < kTok; ++j) {
          const uint4 q = xs[j * nvec + c0 + 32 * u];
          const uint32_t v[4] = {q.x, q.y, q.z, q.w};
          float p = 0.0f;
#pragma unroll
          for (int i = 0; i < 4; ++i) p = fmaf(bf16_hi(v[i]), w[u].hi(i), fmaf(bf16_lo(v[i]), w[u].lo(i), p));
          const float y = p - comp[j], t = s[j] + y;
          comp[j] = (t - s[j]) - y;
          s[j] = t;
        }
      }
    }
#pragma unroll
    for (int j = 0; j < kTok; ++j) {
      double v = static_cast<double>(s[j]) - static_cast<double>(comp[j]);
#pragma unroll
      for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
      if (lane == 0 && j < ntok)
        asm volatile("st.shared::cluster.f64 [%0], %1;" ::"r"(remote + (j * kMoeMaxExperts + e) * 8), "d"(v) : "memory");
    }
  }

  // this CTA's eighth of the token rows, in FP16 times 2^(14 - exponent of the row's largest)
#pragma unroll
  for (int j = 0; j < kTok; ++j) {
    if (j >= ntok) break;
    const int ex = exponent_of(__reduce_max_sync(0xFFFFFFFFu, part[j][lane & (kWarps - 1)]));
    const float up = pow2(14 - ex);
#pragma unroll 1
    for (int c = rank * kThreads + tid; c < nvec; c += kRouteCtas * kThreads) {
      const uint4 q = xs[j * nvec + c];
      const uint32_t v[4] = {q.x, q.y, q.z, q.w};
      uint32_t h[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) h[i] = f16x2_from_f32(bf16_lo(v[i]) * up, bf16_hi(v[i]) * up);
      reinterpret_cast<uint4*>(a.xh + static_cast<long long>(t0 + j) * D)[c] = make_uint4(h[0], h[1], h[2], h[3]);
    }
    if (rank == 0 && tid == 0) a.xscale[t0 + j] = pow2(ex - 14);
  }
  cluster_barrier();
  if (rank != 0 || warp >= ntok) return;

  // top-k of one token by one warp; lane l looks after experts l, l + 32, ...
  const int t = t0 + warp, E = a.E;
  double* sc = score[warp];
  unsigned long long* ks = key[warp];
  double mx = -CUDART_INF, sum = 0.0;
  if (!a.sigmoid) {
#pragma unroll 1
    for (int e = lane; e < E; e += 32) mx = fmax(mx, sc[e]);
#pragma unroll
    for (int o = 16; o; o >>= 1) mx = fmax(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, o));
  }
#pragma unroll 1
  for (int e = lane; e < E; e += 32) {
    const double l = sc[e], ex = exp(a.sigmoid ? -l : l - mx);
    const double p = a.sigmoid ? 1.0 / (1.0 + ex) : ex;
    sum += p;
    sc[e] = p;
    ks[e] = order_key(l);
  }
  double norm = 1.0;
  if (!a.sigmoid) {
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    norm = 1.0 / sum;
  }
  if (a.bias) {
#pragma unroll 1
    for (int e = lane; e < E; e += 32) ks[e] = order_key(sc[e] * norm + static_cast<double>(__ldg(a.bias + e)));
  }
  auto scan = [&](unsigned long long& best, int& at) {
    best = 0;
    at = 0;
#pragma unroll 1
    for (int e = lane; e < E; e += 32) {
      if (ks[e] > best) {                         // ties: the lowest index
        best = ks[e];
        at = e;
      }
    }
  };
  unsigned long long best;
  int at, my_id = 0;
  scan(best, at);
  double wsum = 0.0, mine = 0.0;                  // lane j keeps the j-th weight
#pragma unroll 1
  for (int j = 0; j < a.k; ++j) {
    const uint32_t hi = __reduce_max_sync(0xFFFFFFFFu, static_cast<uint32_t>(best >> 32));
    const uint32_t lo = __reduce_max_sync(0xFFFFFFFFu, static_cast<uint32_t>(best >> 32) == hi ? static_cast<uint32_t>(best) : 0u);
    const bool top = best == ((static_cast<unsigned long long>(hi) << 32) | lo);
    const int id = static_cast<int>(__reduce_min_sync(0xFFFFFFFFu, top ? static_cast<uint32_t>(at) : 0xFFFFFFFFu));
    const double p = sc[id] * norm;
    if (lane == j) {
      mine = p;
      my_id = id;
    }
    wsum += p;
    if (top && at == id) {
      ks[id] = 0;
      scan(best, at);
    }
    __syncwarp();
  }
  const int KT = a.k + a.shared;
  if (lane < KT) {
    float w = 1.0f;
    int id = E + lane - a.k;                      // shared experts follow the routed ones
    if (lane < a.k) {
      w = static_cast<float>((a.renorm ? mine / wsum : mine) * static_cast<double>(a.route_scale));
      id = my_id;
      a.ids[t * a.k + lane] = id;
      a.weights[t * a.k + lane] = w;
    }
    a.pair_id[t * KT + lane] = id;
    a.pair_w[t * KT + lane] = w;
    a.hmax[t * KT + lane] = 0;
  }
}

// ------------------------------------------------------------------ experts' token lists

struct Lists {
  unsigned long long mask[kMoeMaxExperts + kMoeMaxShared];   // tokens of an expert (it has each once)
  uint16_t begin[kMoeMaxExperts + kMoeMaxShared];            // its first place in `pairs`
  uint16_t pairs[kMoeMaxPairs];                              // t * KT + j, grouped by expert
  uint16_t unit[kMoeMaxExperts + kMoeMaxShared + kMoeMaxPairs / 16];   // expert * 4 + its 16 tokens
  int units;
};

// Every CTA groups the (token, expert) pairs by expert for itself.  All find the same order, since
// an expert's units are different CTAs' work.
__device__ __forceinline__ void build_lists(Lists& l, const MoeArgs& a) {
  const int tid = threadIdx.x, n = a.E + a.shared, P = a.T * (a.k + a.shared);
  if (a.T == 1) {                                  // every pair is an expert of its own
    if (tid < P) {
      const int e = __ldcg(a.pair_id + tid);
      l.unit[tid] = static_cast<uint16_t>(e * 4);
      l.pairs[tid] = static_cast<uint16_t>(tid);
      l.begin[e] = static_cast<uint16_t>(tid);
      l.mask[e] = 1;
    }
    if (tid == 0) l.units = P;
    __syncthreads();
    return;
  }
  for (int e = tid; e < n; e += kThreads) l.mask[e] = 0;
  __syncthreads();
  const int KT = a.k + a.shared;
  int id[kMoeMaxPairs / kThreads];
#pragma unroll
  for (int i = 0; i < kMoeMaxPairs / kThreads; ++i) {
    const int q = i * kThreads + tid;
    if (q < P) {
      id[i] = __ldcg(a.pair_id + q);
      // in 32-bit halves, which shared memory does by itself; 64 bits at once are a loop of exchanges
      atomicOr(reinterpret_cast<uint32_t*>(&l.mask[id[i]]) + q / KT / 32, 1u << (q / KT & 31));
    }
  }
  __syncthreads();
  if (tid < 32) {
    int base = 0;                                  // sums of tokens and, 16 bits higher, of units
    for (int e0 = 0; e0 < n; e0 += 32) {
      const int e = e0 + tid, c = e < n ? __popcll(l.mask[e]) : 0, own = c | (c + 15) / 16 << 16;
      int s = own;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xFFFFFFFFu, s, o);
        if (tid >= o) s += v;
      }
      const int before = base + s - own;
      if (e < n) l.begin[e] = static_cast<uint16_t>(before);
      for (int i = 0; i < (c + 15) / 16; ++i) l.unit[(before >> 16) + i] = static_cast<uint16_t>(e * 4 + i);
      base += __shfl_sync(0xFFFFFFFFu, s, 31);
    }
    if (tid == 0) l.units = base >> 16;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kMoeMaxPairs / kThreads; ++i) {
    const int q = i * kThreads + tid;
    if (q < P) l.pairs[l.begin[id[i]] + __popcll(l.mask[id[i]] & ((1ull << (q / KT)) - 1))] = static_cast<uint16_t>(q);
  }
  __syncthreads();
}

// ------------------------------------------------------------------ products

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// A warp's stream of weights: runs of 64 along K of kTiles 8-row tiles, copied to shared
// memory kStages - 1 runs ahead.  A lane reads back only what it copied itself, so the
// stream needs no barriers.  (Held in registers one block ahead, the kernels spilled and the up
// kernel ran at a seventh of the memory rate.)  What shared memory leaves of an SM's 256 KB is
// the L1 that the warps share their activations through, and it counts for more than a deeper
// stream: 64 tokens, 65 experts of 3 x 5120 x 2048, took 437 us with four stages and a second
// buffer of sums (34 KB of L1), 420 without the buffer, 416 with three stages (107 KB); an L2
// prefetch of 256 bytes rather than 128 is worth 441 -> 416.
constexpr int kStages = 3;
constexpr int kRunBytes = kTiles * 512;
constexpr int kStreamBytes = kWarps * kStages * kRunBytes;
__device__ __forceinline__ void cp_async16_or_zero(uint32_t dst, const void* src, bool in) {
  const uint32_t n = in ? 16u : 0u;
  asm volatile("cp.async.cg.shared.global.L2::256B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
  return v;
}

// One 64-element run: the weight tiles at `stage` (this lane's bytes) against eight tokens, and
// against eight more where kWide.  Tiles 2i and 2i + 1 are the 16 rows of one product, so a
// thread gets weight rows g and g + 8 and tokens 2 t and 2 t + 1.
template <bool kWide>
__device__ __forceinline__ void mma_run(float (&b0)[2][4], float (&b1)[2][4], uint32_t stage, const uint32_t (&x0)[8],
                                        const uint32_t (&x1)[8]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint4 wa = lds128(stage + i * 1024), wb = lds128(stage + i * 1024 + 512);
    const uint32_t p[4] = {wa.x, wa.y, wa.z, wa.w}, q[4] = {wb.x, wb.y, wb.z, wb.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t a0 = f16x2_from_e4m3x2(p[j] & 0xFFFFu), a2 = f16x2_from_e4m3x2(p[j] >> 16);
      const uint32_t a1 = f16x2_from_e4m3x2(q[j] & 0xFFFFu), a3 = f16x2_from_e4m3x2(q[j] >> 16);
      mma16816(b0[i], a0, a1, a2, a3, x0[2 * j], x0[2 * j + 1]);
      if (kWide) mma16816(b1[i], a0, a1, a2, a3, x1[2 * j], x1[2 * j + 1]);
    }
  }
}

// 32 bytes into v where `has`; v keeps its zeros elsewhere (no select per register).
__device__ __forceinline__ void load_run(uint32_t (&v)[8], const uint16_t* p, bool has) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %9, 0;\n\t"
      "@q ld.global.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n\t}"
      : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7])
      : "l"(p), "r"(static_cast<uint32_t>(has)));
}

// Scales 16 hidden values, stored relative to the exponents `e` of their two strips of 8, to the row's.
__device__ __forceinline__ void scale_hidden(uint32_t (&v)[8], int2 e, int row_exp) {
  // a strip's exponent is at most the row's; lanes without values have any, and stay zero
  const float f0 = pow2(min(max(e.x - row_exp + 14, -30), 14)), f1 = pow2(min(max(e.y - row_exp + 14, -30), 14));
  const uint32_t h0 = f16x2_from_f32(f0, f0), h1 = f16x2_from_f32(f1, f1);
#pragma unroll
  for (int j = 0; j < 8; ++j) asm("mul.rn.f16x2 %0, %0, %1;" : "+r"(v[j]) : "r"(j < 4 ? h0 : h1));
}

// The products of both layers.  A row group is four tiles: for the up layer the gate and the
// up rows of 16 hidden columns, for the down layer 32 output rows.  A unit is up to 16 tokens of
// an expert, an item a unit and kGroups row groups; kSplit warps share a group's blocks along K
// and meet in shared memory.  The CTAs walk through the items side by side, so that all of them
// read the same few megabytes at a time: with a run of items of its own for each CTA, 1.4 GB of
// experts took twice as long (the pages of 296 places do not fit the address caches).  More
// than 16 tokens of an expert are several units, whose weights all but the first read from L2; as
// further passes of one CTA they left the others waiting at the end (64 tokens with a shared
// expert: 470 -> 437 us).
//
// kOne (down, one token): a cluster of the token's experts owns 64 output rows; the shares meet
// in distributed shared memory and there is no combine kernel.
//
// Measured, device time past L2: 64 tokens, 65 experts of 3 x 5120 x 2048 (2.05 GB): 411 us for
// the layer, 5.0 TB/s of weights, in runs of tens of milliseconds, 450 to 460 us in runs of seconds,
// which the power limit holds at 1.65 GHz; 16 tokens, 23 of 32 and one shared expert of 3 x 4096 x 2048
// (0.60 GB): 127 us, 4.8 TB/s; 64 tokens, all on each of 8 experts of 3 x 5120 x 2048 (0.25 GB, floor
// 39 us): 230 us, four units an expert, whose conversion to FP16 and activations are each unit's own.  Bound by the latency of the loads: 16 warps an SM, each with 4 KB
// of weights on the way, leave the schedulers idle for 60% of the time.  One token, 8 experts of
// 3 x 2048 x 1024: 26 us, of which 14 are there without the weights, in the chain of three kernels:
// 5 us in the router (2.4 of them for the choice), 3 and 2 us in the first pass of the products,
// about twice the time of a second one, since its instructions come from L2.  Passes without
// tokens while the kernel before runs, to have the instructions, won 1 us there and cost 20 at 64
// tokens.
template <bool kUp, int kSplit, bool kOne = false>
__global__ void __launch_bounds__(kThreads, 2)
moe_product_kernel(const __grid_constant__ MoeArgs a) {
  constexpr int kGroups = kWarps / kSplit;
  __shared__ float own[kOne ? 32 * kGroups : 1];
  extern __shared__ __align__(16) uint8_t stream[];
  __shared__ Lists l;
  __shared__ float4 red[2][kWarps][kTiles / 2][32];
  if (kUp) griddep_wait();
  // in the up kernel after the wait: the down kernel may then read the route's results at once
  griddep_launch_dependents();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t4 = lane & 3;
  build_lists(l, a);
  const int K = kUp ? a.D : a.F, F = a.F, D = a.D, KT = a.k + a.shared;
  const int KB = (K + 127) / 128, NB = ((kUp ? 2 * F : D) + 127) / 128;
  const int groups = kUp ? F / 16 : (D + 31) / 32, per = (groups + kGroups - 1) / kGroups;   // items of an expert
  const int items = l.units * per, stride = kOne ? items : static_cast<int>(gridDim.x);
  const int first = kOne ? static_cast<int>(cta_rank()) * per + static_cast<int>(blockIdx.x) / (a.k + a.shared)
                         : static_cast<int>(blockIdx.x);
  const int sub = warp / kSplit, kp = warp % kSplit;
  const int b0 = KB * kp / kSplit, b1 = KB * (kp + 1) / kSplit, runs = 2 * (b1 - b0);
  const uint8_t* const W = kUp ? a.w13 : a.w2;
  const uint16_t* const A = kUp ? a.xh : a.h;

  // ---- the weight stream
  const uint32_t ring = smem_u32(stream) + warp * (kStages * kRunBytes) + lane * 16;
  int ci = first, cr = 0, cslot = 0;
  const uint8_t* cbase = nullptr;
  int o1 = 8 * K, o2 = kUp ? F * K : 16 * K, o3 = o2 + 8 * K;      // offsets of tiles 1 to 3
  auto seek = [&] {
    const int u = ci / per, e = l.unit[u] >> 2, grp = min((ci - u * per) * kGroups + sub, groups - 1);
    const int n = grp * (kUp ? 16 : 32);
    cbase = W + (static_cast<long long>(e) * (kUp ? 2 * F : D) + n + g) * K + b0 * 128 + t4 * 16;
    if (!kUp && n + 32 > D) {                       // the matrix ends inside the group: a tile twice
      o2 = o3 = o1;
    } else if (!kUp) {
      o2 = 16 * K;
      o3 = 24 * K;
    }
  };
  auto copy_run = [&] {
    if (ci < items && runs) {
      const bool in = b0 * 128 + cr * 64 + t4 * 16 < K;
      const uint8_t* src = in ? cbase + cr * 64 : cbase;
      const uint32_t dst = ring + cslot * kRunBytes;
      cp_async16_or_zero(dst, src, in);
      cp_async16_or_zero(dst + 512, src + o1, in);
      cp_async16_or_zero(dst + 1024, src + o2, in);
      cp_async16_or_zero(dst + 1536, src + o3, in);
      if (++cr == runs) {
        cr = 0;
        if ((ci += stride) < items) seek();
      }
    }
    cp_async_commit();
    cslot = cslot + 1 == kStages ? 0 : cslot + 1;
  };
  if (ci < items) seek();
#pragma unroll 1
  for (int i = 0; i < kStages - 1; ++i) copy_run();
  // the down layer's weights do not depend on the kernels before, its activations do
  if (!kUp) griddep_wait();

  int slot = 0;
  // One pass over an item for `cnt` tokens, at most 8 or (kWide) 16.
  auto pass = [&](auto wide_t, int e, int grp0, const uint16_t* pairs, int cnt, int step, bool sync) {
    constexpr bool kWide = decltype(wide_t)::value;
    constexpr int kHalves = kWide ? 2 : 1;
    // this lane's token of either eight, as the products' second operand
    int row[2], rexp[2];
    bool has[2];
#pragma unroll
    for (int h = 0; h < kHalves; ++h) {
      has[h] = h * 8 + g < cnt;
      const int q = has[h] ? pairs[h * 8 + g] : 0;
      row[h] = kUp ? q / KT : q;
      if (!kUp) rexp[h] = exponent_of(__ldcg(a.hmax + q));
    }
    const int n = min(grp0 + sub, groups - 1) * (kUp ? 16 : 32);
    const float* S = (kUp ? a.s13 : a.s2) + (static_cast<long long>(e) * NB + n / 128) * KB;
    const int up_rows = kUp ? ((F + n) / 128 - n / 128) * KB : 0;      // from the gate's scales to the up rows'
    float out[2][2][4];
#pragma unroll
    for (int h = 0; h < kHalves; ++h)
#pragma unroll
      for (int i = 0; i < 2; ++i) out[h][i][0] = out[h][i][1] = out[h][i][2] = out[h][i][3] = 0.0f;
    // Activations, kDepth - 1 runs ahead of the products, and scales two blocks ahead: where the
    // weights have arrived a run takes less than a load from L2 (one token, 8 experts of 3 x 2048 x
    // 1024: 27.2 -> 25.7 us against one run and one block).
    constexpr int kDepth = kWide ? 2 : 4;
    uint32_t x[kDepth][2][8];
    int2 xe[kDepth][2];
#pragma unroll
    for (int c = 0; c < kDepth; ++c)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        xe[c][h] = make_int2(0, 0);
#pragma unroll
        for (int j = 0; j < 8; ++j) x[c][h][j] = 0;
      }
    auto fetch = [&](uint32_t (&v)[2][8], int2 (&ve)[2], int r) {
      const int k = b0 * 128 + r * 64 + t4 * 16;
#pragma unroll
      for (int h = 0; h < kHalves; ++h) {
        if (K & 127) {                                // the last block may end anywhere
#pragma unroll
          for (int j = 0; j < 8; ++j) v[h][j] = 0;
        }
        const bool in = has[h] && k < K;
        load_run(v[h], A + static_cast<long long>(row[h]) * K + k, in);
        if (!kUp && in) ve[h] = __ldcg(reinterpret_cast<const int2*>(a.hexp + (static_cast<long long>(row[h]) * F + k) / 8));
      }
    };
    float s_gate[2] = {0.0f, 0.0f}, s_up[2] = {0.0f, 0.0f};
    auto fetch_scales = [&](int i, int b) {
      s_gate[i] = __ldg(S + b);
      s_up[i] = __ldg(S + b + up_rows);
    };
#pragma unroll
    for (int r = 0; r < kDepth - 1; ++r)
      if (r < runs) fetch(x[r], xe[r], r);
    if (runs) fetch_scales(0, b0);
    if (b0 + 1 < b1) fetch_scales(1, b0 + 1);
#pragma unroll 1
    for (int b = b0; b < b1; b += kDepth / 2) {
#pragma unroll
      for (int u = 0; u < kDepth / 2; ++u) {
        if (b + u >= b1) break;
        float k0[2][4], k1[2][4];
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) k0[i][j] = k1[i][j] = 0.0f;
#pragma unroll
        for (int v = 0; v < 2; ++v) {
          const int c = 2 * u + v, r = 2 * (b - b0) + c;
          constexpr int kAhead = kDepth - 1;
          if (r + kAhead < runs) fetch(x[(c + kAhead) % kDepth], xe[(c + kAhead) % kDepth], r + kAhead);
          if (!kUp) {
#pragma unroll
            for (int h = 0; h < kHalves; ++h) scale_hidden(x[c][h], xe[c][h], rexp[h]);
          }
          cp_async_wait<kStages - 2>();
          mma_run<kWide>(k0, k1, ring + slot * kRunBytes, x[c][0], x[c][1]);
          copy_run();                       // into the slot before this one, read by now
          slot = slot + 1 == kStages ? 0 : slot + 1;
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            out[0][i][j] = fmaf(k0[i][j], i ? s_up[0] : s_gate[0], out[0][i][j]);
            if (kWide) out[1][i][j] = fmaf(k1[i][j], i ? s_up[0] : s_gate[0], out[1][i][j]);
          }
        s_gate[0] = s_gate[1];
        s_up[0] = s_up[1];
        if (b + u + 2 < b1) fetch_scales(1, b + u + 2);
      }
    }
    if (sync) __syncthreads();
#pragma unroll
    for (int h = 0; h < kHalves; ++h)
#pragma unroll
      for (int i = 0; i < 2; ++i)
        red[(step + h) & 1][warp][i][lane] = make_float4(out[h][i][0], out[h][i][1], out[h][i][2], out[h][i][3]);
    __syncthreads();
    if (kUp) {
      // a warp (in turn) for each group and eight tokens: product 0 are the gate rows, product 1 the up rows
      const int task = (warp - 2 * kGroups * step) & (kWarps - 1), grp = task >> 1, h = task & 1;
      if (grp < kGroups && h < kHalves && grp0 + grp < groups) {
        float gs[4] = {0, 0, 0, 0}, us[4] = {0, 0, 0, 0};
#pragma unroll
        for (int w = 0; w < kSplit; ++w) {
          const float4 p = red[(step + h) & 1][grp * kSplit + w][0][lane], q = red[(step + h) & 1][grp * kSplit + w][1][lane];
          gs[0] += p.x; gs[1] += p.y; gs[2] += p.z; gs[3] += p.w;
          us[0] += q.x; us[1] += q.y; us[2] += q.z; us[3] += q.w;
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {                   // tokens 2 t and 2 t + 1
          const int r = h * 8 + 2 * t4 + j, q = r < cnt ? pairs[r] : 0;
          const float xs = r < cnt ? a.xscale[q / KT] : 0.0f;
          int top = 0;
#pragma unroll
          for (int i = 0; i < 2; ++i) {                 // hidden columns f + g, for each eight of the group's 16
            const float gv = gs[2 * i + j] * xs, uv = us[2 * i + j] * xs;
            const float v = gv / (1.0f + expf(-gv)) * uv;
            int m = static_cast<int>(__float_as_uint(v) & 0x7FFFFFFFu);
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
            const int ex = exponent_of(m), f = (grp0 + grp) * 16 + i * 8;
            top = max(top, m);
            if (r < cnt) {
              a.h[static_cast<long long>(q) * F + f + g] =
                  static_cast<uint16_t>(f16x2_from_f32(0.5f * v * pow2(1 - ex), 0.0f));
              if (g == 0) a.hexp[static_cast<long long>(q) * (F / 8) + f / 8] = ex;
            }
          }
          if (r < cnt && g == 0) atomicMax(a.hmax + q, static_cast<uint32_t>(top));
        }
      }
    } else {
      // task (group, eight tokens, product): the sums of the group's kSplit warps
#pragma unroll
      for (int task = warp; task < 4 * kGroups; task += kWarps) {
        const int grp = task >> 2, h = (task >> 1) & 1, i = task & 1, row = (grp0 + grp) * 32 + i * 16 + g;
        if (h >= kHalves) continue;
        float v[4] = {0, 0, 0, 0};
#pragma unroll
        for (int w = 0; w < kSplit; ++w) {
          const float4 p = red[(step + h) & 1][grp * kSplit + w][i][lane];
          v[0] += p.x; v[1] += p.y; v[2] += p.z; v[3] += p.w;
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int r = h * 8 + 2 * t4 + j;
          if (r < cnt) {
            const int q = pairs[r];
            const float w = __ldcg(a.pair_w + q) * pow2(exponent_of(__ldcg(a.hmax + q)) - 14);
            if (kOne) {
              own[grp * 32 + i * 16 + g] = w * v[j];
              own[grp * 32 + i * 16 + g + 8] = w * v[2 + j];
            } else {
              float* y = a.share + static_cast<long long>(q) * D + row;
              if (row < D) y[0] = w * v[j];
              if (row + 8 < D) y[8] = w * v[2 + j];
            }
          }
        }
      }
    }
  };
  bool wide = false;
  for (int it = first, step = 0; it < items; it += stride, ++step) {
    const int at = it / per, u = l.unit[at], e = u >> 2, p0 = (u & 3) * 16, grp0 = (it - at * per) * kGroups;
    const int cnt = min(16, __popcll(l.mask[e]) - p0);
    const uint16_t* pairs = l.pairs + l.begin[e] + p0;
    // Two buffers of eight tokens' sums: the barrier of the step between orders a buffer's next
    // use after its reads, unless one of the two steps uses both.
    const bool sync = cnt > 8 || wide;
    wide = cnt > 8;
    if (wide) pass(std::true_type(), e, grp0, pairs, cnt, step, sync);
    else pass(std::false_type(), e, grp0, pairs, cnt, step, sync);
  }
  if (kOne) {
    cluster_barrier();
    const int row = (first % per) * 32 * kGroups + tid;
    if (cta_rank() == 0 && tid < 32 * kGroups && row < D) {
      const uint32_t at = smem_u32(own + tid);
      float v[8], sum = 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j < KT) asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v[j]) : "r"(mapa_u32(at, j)));
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j < KT) sum += v[j];
      a.y[row] = static_cast<uint16_t>(bf16x2_from_f32(sum, 0.0f));
    }
    cluster_barrier();             // the first CTA may still be reading this one's sums
  }
}

// ------------------------------------------------------------------ combine

// y[t] = the sum of its pairs' shares, in order; four columns a thread.
__global__ void __launch_bounds__(kThreads)
moe_combine_kernel(const __grid_constant__ MoeArgs a) {
  griddep_launch_dependents();
  griddep_wait();
  const int KT = a.k + a.shared, quads = a.D / 4, i = static_cast<int>(blockIdx.x) * kThreads + threadIdx.x;
  if (i >= a.T * quads) return;
  const int t = i / quads, c = i % quads;
  const float4* p = reinterpret_cast<const float4*>(a.share + static_cast<long long>(t) * KT * a.D) + c;
  float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
  for (int j = 0; j < KT; ++j) {
    const float4 v = __ldcg(p + static_cast<long long>(j) * quads);
    s.x += v.x; s.y += v.y; s.z += v.z; s.w += v.w;
  }
  *reinterpret_cast<uint2*>(a.y + static_cast<long long>(t) * a.D + c * 4) =
      make_uint2(bf16x2_from_f32(s.x, s.y), bf16x2_from_f32(s.z, s.w));
}

size_t align256(size_t v) { return (v + 255) / 256 * 256; }

// Per device: shared-memory limits raised once.
constexpr int kMaxDevices = 64;
struct MoeSetup {
  std::once_flag once;
  cudaError_t err = cudaSuccess;
};

// How many warps share a row group's K.  With few, an item is larger and its barrier and
// joining cost less per byte; with many, the items deal out more evenly over the CTAs.  The
// estimate, in units of a warp's time for one block of 128: a warp's blocks plus 1.5 for the
// end of an item, times the rounds of items plus one.  Measured, us of a whole layer with 8, 4, 2
// warps in the up kernel: 435, 416, 437 (64 tokens, 65 experts of 3 x 5120 x 2048), 94, 81, 81
// (16 tokens, 64 of 3 x 2048 x 1024), 26.5, 28.5, 28 (one token, 8 of 3 x 2048 x 1024); with 4, 2
// in the down kernel 430, 416 and 85, 81.
template <bool kUp>
cudaError_t launch_product(const MoeArgs& a, int units, cudaStream_t s) {
  const long long slots = 2LL * num_sms();
  const int KB = ((kUp ? a.D : a.F) + 127) / 128, groups = kUp ? a.F / 16 : (a.D + 31) / 32;
  int best = 8;
  double cost = 0.0;
  long long best_items = 0;
  for (int split = 8; split >= 2; split /= 2) {
    const int per = (groups + kWarps / split - 1) / (kWarps / split);
    const long long items = static_cast<long long>(units) * per;
    const double c = ((items + slots - 1) / slots + 1.0) * ((KB + split - 1) / split + 1.5);
    if (split == 8 || c < cost) {
      best = split;
      cost = c;
      best_items = items;
    }
  }
  const unsigned grid = static_cast<unsigned>(std::min(slots, best_items));
  if (best == 8) return launch_pdl(moe_product_kernel<kUp, 8>, grid, kThreads, kStreamBytes, 1, s, a);
  if (best == 4) return launch_pdl(moe_product_kernel<kUp, 4>, grid, kThreads, kStreamBytes, 1, s, a);
  return launch_pdl(moe_product_kernel<kUp, 2>, grid, kThreads, kStreamBytes, 1, s, a);
}

}  // namespace

size_t moe_carve(MoeArgs& a, uint8_t* base) {
  const size_t P = static_cast<size_t>(a.T) * (a.k + a.shared);
  size_t at = 0;
  auto take = [&](auto*& p, size_t bytes) {
    p = reinterpret_cast<std::remove_reference_t<decltype(p)>>(base + at);
    at += align256(bytes);
  };
  take(a.pair_id, P * 4);
  take(a.pair_w, P * 4);
  take(a.hmax, P * 4);
  take(a.hexp, P * (a.F / 8) * 4);
  take(a.xh, static_cast<size_t>(a.T) * a.D * 2);
  take(a.xscale, static_cast<size_t>(a.T) * 4);
  take(a.h, P * a.F * 2);
  take(a.share, P * a.D * 4);
  return at;
}

cudaError_t launch_fp8_moe(MoeArgs& a, cudaStream_t s) {
  static MoeSetup setups[kMaxDevices];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= kMaxDevices) return cudaErrorInvalidDevice;
  MoeSetup& d = setups[dev];
  std::call_once(d.once, [&] {
    auto raise = [&](auto* kernel, int bytes) {
      if (d.err == cudaSuccess) d.err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    };
    raise(moe_route_kernel<1, false>, BILOCO_MOE_MAX_D * 2);
    raise(moe_route_kernel<1, true>, BILOCO_MOE_MAX_D * 2);
    raise(moe_route_kernel<2, false>, 2 * BILOCO_MOE_MAX_D * 2);
    raise(moe_route_kernel<2, true>, 2 * BILOCO_MOE_MAX_D * 2);
    raise(moe_product_kernel<true, 8>, kStreamBytes);
    raise(moe_product_kernel<true, 4>, kStreamBytes);
    raise(moe_product_kernel<true, 2>, kStreamBytes);
    raise(moe_product_kernel<false, 8>, kStreamBytes);
    raise(moe_product_kernel<false, 4>, kStreamBytes);
    raise(moe_product_kernel<false, 2>, kStreamBytes);
    raise(moe_product_kernel<false, 4, true>, kStreamBytes);
  });
  if (d.err != cudaSuccess) return d.err;

  // Up to 32 tokens a cluster each; above, two share a cluster's reads of the router.  Measured, us of
  // a layer with little else to do (F = 16) with 1, 2, 4 tokens a cluster: 37, 39, 42 (16 x 4096, 64
  // experts), 44, 46, 51 (32 x 4096), 66, 64, 68 (64 x 5120), 96, 92, 96 (64 x 2048, 512 experts).
  const int tok = a.T <= 32 ? 1 : 2;
  const unsigned grid = static_cast<unsigned>((a.T + tok - 1) / tok * kRouteCtas);
  const size_t sm = static_cast<size_t>(tok) * a.D * 2;
  if (tok == 1)
    e = a.router_f32 ? launch_pdl(moe_route_kernel<1, true>, grid, kThreads, sm, kRouteCtas, s, a)
                     : launch_pdl(moe_route_kernel<1, false>, grid, kThreads, sm, kRouteCtas, s, a);
  else
    e = a.router_f32 ? launch_pdl(moe_route_kernel<2, true>, grid, kThreads, sm, kRouteCtas, s, a)
                     : launch_pdl(moe_route_kernel<2, false>, grid, kThreads, sm, kRouteCtas, s, a);
  if (e != cudaSuccess) return e;

  const int units = std::min(a.T * a.k, a.E) + a.shared * ((a.T + 15) / 16);     // about
  e = launch_product<true>(a, units, s);
  if (e != cudaSuccess) return e;
  if (a.T == 1 && a.k + a.shared <= 8) {
    const unsigned n = static_cast<unsigned>(a.k + a.shared);
    return launch_pdl(moe_product_kernel<false, 4, true>, static_cast<unsigned>((a.D + 63) / 64) * n, kThreads, kStreamBytes, n,
                      s, a);
  }
  e = launch_product<false>(a, units, s);
  if (e != cudaSuccess) return e;
  return launch_pdl(moe_combine_kernel, static_cast<unsigned>((a.T * (a.D / 4) + kThreads - 1) / kThreads), kThreads, 0, 1,
                    s, a);
}

}  // namespace biloco
