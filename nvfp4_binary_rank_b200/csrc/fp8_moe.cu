// A whole mixture-of-experts layer for a few tokens, with FP8 block-scaled experts:
//
//   scores = x router^T;  the k best experts of each token, weights w from softmax or sigmoid
//   y[t] = sum over its experts e of w_e * W2_e (silu(W1_e x) * (W3_e x)),  W13 = [W1; W3]
//
// With few tokens the layer is the stream of the picked experts' weights: 3 D F bytes for
// each of them, everything else is small.  So every weight byte is read once, straight into
// the registers that feed the multiplication (a warp's 16-byte loads cover eight rows of 64
// bytes), and the tokens of an expert share it.  The products run on the warp-level tensor
// instruction (m16n8k16, FP16 operands, FP32 sums): at up to 16 tokens per expert it needs
// about a third of its rate, where a tcgen05 tile would first have to go through shared
// memory.  E4M3 values are exact in FP16.  The activations are not quantised: a token's row
// is scaled by a power of two into FP16's range, which is exact for BF16 values down to
// 2^-29 of the row's largest, and the hidden row keeps FP16's 11 bits.
//
// Within a block of 128 along K the order of the terms is free, so lane t of a quad takes 16
// consecutive elements of a 64-element run for both operands and no data is exchanged.
//
// Three kernels on one stream, each launched while the one before it ends:
//   route  scores in FP32 with compensated sums, top-k, the token rows in FP16
//   up     per (expert, 16 hidden columns): gate and up rows over the whole of D, split
//          over the CTA's warps; h as FP16 with a scale per 16 columns and the row's maximum
//   down   per 32 output rows: all experts' h; the (expert, block) units are dealt out
//          evenly over a cluster's warps, whose sums are added in a fixed order
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
// 2^(14 - e) and 2^(e - 14) are normal numbers.
__device__ __forceinline__ int exponent_of(uint32_t bits) {
  return min(max(static_cast<int>(bits >> 23) - 127, -100), 127);
}

// ------------------------------------------------------------------ route

template <bool kF32>
__device__ __forceinline__ void load_router8(const void* p, long long at, float (&v)[8]) {
  if (kF32) {
    const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(p) + at);
    const float4 a = __ldg(q), b = __ldg(q + 1);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  } else {
    const uint4 a = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + at));
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[2 * j] = bf16_lo(w[j]);
      v[2 * j + 1] = bf16_hi(w[j]);
    }
  }
}

// A cluster of eight CTAs serves kTok tokens: each CTA scores an eighth of the experts for
// all of them (the router is read once per cluster), the first one picks.
template <int kTok, bool kF32>
__global__ void __launch_bounds__(kThreads)
moe_route_kernel(const __grid_constant__ MoeArgs a) {
  extern __shared__ __align__(16) uint8_t sm[];
  uint16_t* xs = reinterpret_cast<uint16_t*>(sm);                       // [kTok][D] bf16
  __shared__ double logits[kTok][kMoeMaxExperts];
  __shared__ uint32_t part[kTok][kWarps];
  griddep_launch_dependents();
  griddep_wait();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = static_cast<int>(cta_rank());
  const int t0 = static_cast<int>(blockIdx.x) / kRouteCtas * kTok;
  const int D = a.D, nvec = D / 8;

  // the token rows into shared memory, and each row's largest magnitude
  uint32_t top[kTok];
#pragma unroll
  for (int j = 0; j < kTok; ++j) {
    top[j] = 0;
    if (t0 + j < a.T) {
      for (int c = tid; c < nvec; c += kThreads) {
        const uint4 q = __ldg(reinterpret_cast<const uint4*>(a.x + (t0 + j) * a.ldx) + c);
        reinterpret_cast<uint4*>(xs + j * D)[c] = q;
        const uint32_t m = __vmaxu2(__vmaxu2(q.x & 0x7FFF7FFFu, q.y & 0x7FFF7FFFu),
                                    __vmaxu2(q.z & 0x7FFF7FFFu, q.w & 0x7FFF7FFFu));
        top[j] = max(top[j], max(m << 16, m & 0xFFFF0000u));
      }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) top[j] = max(top[j], __shfl_xor_sync(0xFFFFFFFFu, top[j], o));
    if (lane == 0) part[j][warp] = top[j];
  }
  cluster_barrier();                // also: the first CTA runs, so its shared memory may be written

  // scores: a warp takes whole experts; sums of eight products, compensated over a lane's
  // eights (Kahan), in FP64 over the lanes
  const uint32_t remote = mapa_u32(smem_u32(&logits[0][0]), 0);
  for (int e = rank + kRouteCtas * warp; e < a.E; e += kRouteCtas * kWarps) {
    float s[kTok], comp[kTok];
#pragma unroll
    for (int j = 0; j < kTok; ++j) s[j] = comp[j] = 0.0f;
#pragma unroll 2
    for (int c = lane; c < nvec; c += 32) {
      float w[8];
      load_router8<kF32>(a.router, static_cast<long long>(e) * D + c * 8, w);
#pragma unroll
      for (int j = 0; j < kTok; ++j) {
        if (t0 + j >= a.T) break;
        const uint4 q = reinterpret_cast<const uint4*>(xs + j * D)[c];
        const uint32_t x[4] = {q.x, q.y, q.z, q.w};
        float p = 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i) p = fmaf(bf16_hi(x[i]), w[2 * i + 1], fmaf(bf16_lo(x[i]), w[2 * i], p));
        const float y = p - comp[j], t = s[j] + y;
        comp[j] = (t - s[j]) - y;
        s[j] = t;
      }
    }
#pragma unroll
    for (int j = 0; j < kTok; ++j) {
      double v = static_cast<double>(s[j]) - static_cast<double>(comp[j]);
#pragma unroll
      for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
      if (lane == 0)
        asm volatile("st.shared::cluster.f64 [%0], %1;" ::"r"(remote + (j * kMoeMaxExperts + e) * 8), "d"(v) : "memory");
    }
  }

  // this CTA's eighth of the token rows, in FP16 times 2^(14 - exponent of the largest)
#pragma unroll
  for (int j = 0; j < kTok; ++j) {
    if (t0 + j >= a.T) break;
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) m = max(m, part[j][i]);
    const int ex = exponent_of(m);
    const float up = pow2(14 - ex);
    for (int c = rank * kThreads + tid; c < nvec; c += kRouteCtas * kThreads) {
      const uint4 q = reinterpret_cast<const uint4*>(xs + j * D)[c];
      const uint32_t x[4] = {q.x, q.y, q.z, q.w};
      uint32_t h[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) h[i] = f16x2_from_f32(bf16_lo(x[i]) * up, bf16_hi(x[i]) * up);
      reinterpret_cast<uint4*>(a.xh + static_cast<long long>(t0 + j) * D)[c] = make_uint4(h[0], h[1], h[2], h[3]);
    }
    if (rank == 0 && tid == 0) a.xscale[t0 + j] = pow2(ex - 14);
  }
  cluster_barrier();
  if (rank != 0 || warp >= kTok || t0 + warp >= a.T) return;

  // top-k of one token by one warp: keys and scores in FP64, lane l holds experts l, l + 32, ...
  constexpr int kPer = kMoeMaxExperts / 32;
  const int t = t0 + warp;
  double key[kPer], p[kPer];
  const double kNone = -CUDART_INF;
  double mx = kNone;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = i * 32 + lane;
    p[i] = e < a.E ? logits[warp][e] : kNone;
    mx = fmax(mx, p[i]);
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) mx = fmax(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, o));
  double sum = 0.0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = i * 32 + lane;
    if (i * 32 >= a.E) break;
    const double l = p[i];
    if (a.sigmoid) {
      p[i] = 1.0 / (1.0 + exp(-l));
    } else {
      p[i] = e < a.E ? exp(l - mx) : 0.0;
      sum += p[i];
    }
    key[i] = a.bias ? 0.0 : l;
  }
  if (!a.sigmoid) {
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
  }
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = i * 32 + lane;
    if (i * 32 >= a.E) break;
    if (!a.sigmoid) p[i] /= sum;
    if (e < a.E && a.bias) key[i] = p[i] + static_cast<double>(__ldg(a.bias + e));
    if (isnan(key[i])) key[i] = kNone;            // a score that is no number is picked last
  }
  uint32_t used = 0;
  double wsum = 0.0, mine = 0.0;                  // lane j keeps the j-th weight
  int my_id = 0;
  for (int j = 0; j < a.k; ++j) {
    double best = kNone, bp = 0.0;
    int bi = 0x7FFFFFFF;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int e = i * 32 + lane;
      if (e < a.E && !(used >> i & 1) && (bi == 0x7FFFFFFF || key[i] > best)) {
        best = key[i];
        bi = e;
        bp = p[i];
      }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) {                // ties: the lowest index
      const double ob = __shfl_xor_sync(0xFFFFFFFFu, best, o), op = __shfl_xor_sync(0xFFFFFFFFu, bp, o);
      const int oi = __shfl_xor_sync(0xFFFFFFFFu, bi, o);
      if (oi != 0x7FFFFFFF && (bi == 0x7FFFFFFF || ob > best || (ob == best && oi < bi))) {
        best = ob;
        bi = oi;
        bp = op;
      }
    }
    if ((bi & 31) == lane) used |= 1u << (bi >> 5);
    if (lane == j) {
      mine = bp;
      my_id = bi;
    }
    wsum += bp;
  }
  const int KT = a.k + a.shared;
  if (lane < KT) {
    float w = 1.0f;
    int id = a.E + lane - a.k;                    // shared experts follow the routed ones
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
  int count[kMoeMaxExperts + kMoeMaxShared];       // tokens of an expert
  int begin[kMoeMaxExperts + kMoeMaxShared];       // its first place in `pairs`
  int active[kMoeMaxExperts + kMoeMaxShared];      // experts with tokens, ascending
  int pairs[kMoeMaxPairs];                         // t * KT + j, grouped by expert
  int nact;
};

// Every CTA groups the (token, expert) pairs by expert for itself.
__device__ __forceinline__ void build_lists(Lists& l, const MoeArgs& a) {
  const int tid = threadIdx.x, n = a.E + a.shared, P = a.T * (a.k + a.shared);
  for (int e = tid; e < n; e += kThreads) l.count[e] = 0;
  __syncthreads();
  int pos[kMoeMaxPairs / kThreads], id[kMoeMaxPairs / kThreads];
#pragma unroll
  for (int i = 0; i < kMoeMaxPairs / kThreads; ++i) {
    const int q = i * kThreads + tid;
    if (q < P) {
      id[i] = __ldcg(a.pair_id + q);
      pos[i] = atomicAdd(&l.count[id[i]], 1);
    }
  }
  __syncthreads();
  if (tid < 32) {
    int base = 0, na = 0;
    for (int e0 = 0; e0 < n; e0 += 32) {
      const int e = e0 + tid, c = e < n ? l.count[e] : 0;
      int s = c;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xFFFFFFFFu, s, o);
        if (tid >= o) s += v;
      }
      const uint32_t has = __ballot_sync(0xFFFFFFFFu, c > 0);
      if (e < n) l.begin[e] = base + s - c;
      if (c > 0) l.active[na + __popc(has & ((1u << tid) - 1))] = e;
      base += __shfl_sync(0xFFFFFFFFu, s, 31);
      na += __popc(has);
    }
    if (tid == 0) l.nact = na;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kMoeMaxPairs / kThreads; ++i)
    if (i * kThreads + tid < P) l.pairs[l.begin[id[i]] + pos[i]] = i * kThreads + tid;
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

// The weight bytes of one block of 128 along K: two 64-element runs of kTiles 8-row tiles.
struct WBlock {
  uint4 w[2][kTiles];
};
__device__ __forceinline__ uint4 ld_weight(const uint8_t* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}
// `row[i]`: this lane's row of tile i, or null past the matrix.
__device__ __forceinline__ void load_wblock(WBlock& b, const uint8_t* const (&row)[kTiles], int k, int K) {
#pragma unroll
  for (int c = 0; c < 2; ++c)
#pragma unroll
    for (int i = 0; i < kTiles; ++i)
      b.w[c][i] = (row[i] && k + c * 64 < K) ? ld_weight(row[i] + k + c * 64) : make_uint4(0, 0, 0, 0);
}

// blk[i] += tokens x tile i over one 64-element run; lo/hi: 16 FP16 values of token rows g, g + 8.
__device__ __forceinline__ void mma_run(float (&blk)[kTiles][4], const uint4 (&w)[kTiles], const uint32_t (&lo)[8],
                                        const uint32_t (&hi)[8]) {
#pragma unroll
  for (int i = 0; i < kTiles; ++i) {
    const uint32_t q[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
    for (int j = 0; j < 4; ++j)
      mma16816(blk[i], lo[2 * j], hi[2 * j], lo[2 * j + 1], hi[2 * j + 1], f16x2_from_e4m3x2(q[j] & 0xFFFFu),
               f16x2_from_e4m3x2(q[j] >> 16));
  }
}

__device__ __forceinline__ void load_row16(uint32_t (&v)[8], const uint16_t* p) {
  if (p) {
    const uint4 a = *reinterpret_cast<const uint4*>(p), b = *(reinterpret_cast<const uint4*>(p) + 1);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = 0;
  }
}

// ------------------------------------------------------------------ up

// Item (expert, 16 hidden columns): two tiles of gate rows, the two tiles of the same up
// rows.  The CTA's warps split D; their sums meet in shared memory, where one warp at a time
// finishes an item while the others go on.  Items of one expert follow each other in a CTA,
// so its token rows stay in L1.  More than 16 tokens of an expert take further passes over
// the item's weights, which then come from L2.
__global__ void __launch_bounds__(kThreads, 2)
moe_up_kernel(const __grid_constant__ MoeArgs a) {
  __shared__ Lists l;
  __shared__ float4 red[2][kWarps][kTiles][32];
  griddep_wait();
  griddep_launch_dependents();      // after the wait: the next kernel may read the route's results at once
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t4 = lane & 3;
  build_lists(l, a);
  const int D = a.D, F = a.F, KT = a.k + a.shared;
  const int KB = (D + 127) / 128, NB = (2 * F + 127) / 128, strips = F / 16;
  const int items = l.nact * strips;
  const int b0 = KB * warp / kWarps, b1 = KB * (warp + 1) / kWarps;
  int it = static_cast<int>(static_cast<long long>(items) * blockIdx.x / gridDim.x);
  const int it1 = static_cast<int>(static_cast<long long>(items) * (blockIdx.x + 1) / gridDim.x);
  const uint8_t* row[kTiles];
  // tile i: gate (0, 1) or up (2, 3) rows; a tile never crosses a block of 128 rows
  auto tile_row = [&](int item, int i) { return (i >> 1) * F + item % strips * 16 + (i & 1) * 8; };
  auto set_rows = [&](int item) {
    const uint8_t* W = a.w13 + static_cast<long long>(l.active[item / strips]) * 2 * F * D;
#pragma unroll
    for (int i = 0; i < kTiles; ++i) row[i] = W + static_cast<long long>(tile_row(item, i) + g) * D + t4 * 16;
  };
  WBlock next;
  if (it < it1 && b0 < b1) {
    set_rows(it);
    load_wblock(next, row, b0 * 128, D - t4 * 16);
  }
  for (int p0 = 0, step = 0; it < it1; ++step) {
    const int e = l.active[it / strips], f0 = it % strips * 16;
    const int cnt = min(16, l.count[e] - p0);
    const int* pairs = l.pairs + l.begin[e] + p0;
    const bool more = p0 + 16 < l.count[e];
    const int it_next = more ? it : it + 1;
    const uint16_t* xlo = g < cnt ? a.xh + static_cast<long long>(pairs[g] / KT) * D + t4 * 16 : nullptr;
    const uint16_t* xhi = g + 8 < cnt ? a.xh + static_cast<long long>(pairs[g + 8] / KT) * D + t4 * 16 : nullptr;
    const float* S = a.s13 + static_cast<long long>(e) * NB * KB;
    const float* srow[kTiles];
#pragma unroll
    for (int i = 0; i < kTiles; ++i) srow[i] = S + tile_row(it, i) / 128 * KB;
    float out[kTiles][4];
#pragma unroll
    for (int i = 0; i < kTiles; ++i) out[i][0] = out[i][1] = out[i][2] = out[i][3] = 0.0f;
    for (int b = b0; b < b1; ++b) {
      const WBlock cur = next;
      if (b + 1 < b1) {
        load_wblock(next, row, (b + 1) * 128, D - t4 * 16);
      } else if (it_next < it1) {
        set_rows(it_next);
        load_wblock(next, row, b0 * 128, D - t4 * 16);
      }
      float blk[kTiles][4], s[kTiles];
#pragma unroll
      for (int i = 0; i < kTiles; ++i) {
        blk[i][0] = blk[i][1] = blk[i][2] = blk[i][3] = 0.0f;
        s[i] = __ldg(srow[i] + b);
      }
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int k = b * 128 + c * 64;
        const bool in = k + t4 * 16 < D;
        uint32_t lo[8], hi[8];
        load_row16(lo, in && xlo ? xlo + k : nullptr);
        load_row16(hi, in && xhi ? xhi + k : nullptr);
        mma_run(blk, cur.w[c], lo, hi);
      }
#pragma unroll
      for (int i = 0; i < kTiles; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) out[i][j] = fmaf(blk[i][j], s[i], out[i][j]);
    }
    // Two buffers: the barrier of the step between orders a buffer's next use after its reads.
    float4(*sums)[kTiles][32] = red[step & 1];
#pragma unroll
    for (int i = 0; i < kTiles; ++i) sums[warp][i][lane] = make_float4(out[i][0], out[i][1], out[i][2], out[i][3]);
    __syncthreads();
    if (warp == (step & (kWarps - 1))) {
      float v[2][4];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float gs[4] = {0, 0, 0, 0}, us[4] = {0, 0, 0, 0};
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          const float4 p = sums[w][i][lane], q = sums[w][2 + i][lane];
          gs[0] += p.x; gs[1] += p.y; gs[2] += p.z; gs[3] += p.w;
          us[0] += q.x; us[1] += q.y; us[2] += q.z; us[3] += q.w;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int r = g + (j >> 1) * 8;
          const float xs = r < cnt ? a.xscale[pairs[r] / KT] : 0.0f;
          const float gv = gs[j] * xs, uv = us[j] * xs;
          v[i][j] = gv / (1.0f + expf(-gv)) * uv;
        }
      }
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int r = g + half * 8;
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int j = 0; j < 2; ++j) m = max(m, __float_as_uint(v[i][half * 2 + j]) & 0x7FFFFFFFu);
        m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
        m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
        if (r < cnt) {
          const int q = pairs[r], ex = exponent_of(m);
          const float up = pow2(-ex);
          uint32_t* h = reinterpret_cast<uint32_t*>(a.h + static_cast<long long>(q) * F + f0 + 2 * t4);
          h[0] = f16x2_from_f32(v[0][half * 2] * up, v[0][half * 2 + 1] * up);
          h[4] = f16x2_from_f32(v[1][half * 2] * up, v[1][half * 2 + 1] * up);
          if (t4 == 0) {
            a.hexp[static_cast<long long>(q) * strips + f0 / 16] = ex;
            atomicMax(a.hmax + q, m);
          }
        }
      }
    }
    p0 = more ? p0 + 16 : 0;
    it = it_next;
  }
}

// ------------------------------------------------------------------ down

// 16 hidden values of pair q from column k (one strip), brought to the row's exponent.
__device__ __forceinline__ void load_hidden(uint32_t (&v)[8], const MoeArgs& a, int q, int k, int row_exp, int strips) {
  if (q < 0) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = 0;
    return;
  }
  const uint4* p = reinterpret_cast<const uint4*>(a.h + static_cast<long long>(q) * a.F + k);
  const uint4 x = __ldcg(p), y = __ldcg(p + 1);
  const int d = max(__ldcg(a.hexp + static_cast<long long>(q) * strips + k / 16) - row_exp + 14, -30);
  const uint32_t f = f16x2_from_f32(pow2(d), pow2(d));
  const uint32_t w[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
#pragma unroll
  for (int j = 0; j < 8; ++j) asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(v[j]) : "r"(w[j]), "r"(f));
}

// A cluster of `a.split` CTAs owns 32 output rows.  Unit (active expert, block of 128 along
// F); a warp takes a run of units and adds each expert's weighted sums into its own
// [tokens][32] array; the arrays are summed over warps and CTAs in order.
__global__ void __launch_bounds__(kThreads, 2)
moe_down_kernel(const __grid_constant__ MoeArgs a) {
  extern __shared__ __align__(16) float acc[];                 // [kWarps][T][kPitch]
  constexpr int kRows = 8 * kTiles, kPitch = kRows + 1;
  __shared__ Lists l;
  griddep_launch_dependents();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t4 = lane & 3;
  const int rank = a.split > 1 ? static_cast<int>(cta_rank()) : 0;
  const int D = a.D, F = a.F, T = a.T, KT = a.k + a.shared;
  const int KB = (F + 127) / 128, NB = (D + 127) / 128, strips = F / 16;
  const int n0 = static_cast<int>(blockIdx.x) / a.split * kRows;
  for (int i = tid; i < kWarps * T * kPitch; i += kThreads) acc[i] = 0.0f;
  build_lists(l, a);                        // the route kernel ended before this one could start
  float* mine = acc + warp * T * kPitch;

  const int units = l.nact * KB, parts = a.split * kWarps, part = rank * kWarps + warp;
  int u = static_cast<int>(static_cast<long long>(units) * part / parts);
  const int u1 = static_cast<int>(static_cast<long long>(units) * (part + 1) / parts);
  const uint8_t* row[kTiles];
  auto set_rows = [&](int unit) {
    const uint8_t* W = a.w2 + static_cast<long long>(l.active[unit / KB]) * D * F;
#pragma unroll
    for (int i = 0; i < kTiles; ++i) {
      const int n = n0 + i * 8 + g;
      row[i] = n < D ? W + static_cast<long long>(n) * F + t4 * 16 : nullptr;
    }
  };
  // the weights do not depend on the kernels before: the first block is requested at once
  WBlock next;
  if (u < u1) {
    set_rows(u);
    load_wblock(next, row, u % KB * 128, F - t4 * 16);
  }
  griddep_wait();
  for (int p0 = 0; u < u1;) {
    const int e = l.active[u / KB], ba = u % KB, bb = min(KB, ba + u1 - u);
    const int cnt = min(16, l.count[e] - p0);
    const int* pairs = l.pairs + l.begin[e] + p0;
    const bool more = p0 + 16 < l.count[e];
    const int u_next = more ? u : u + bb - ba;
    const float* S = a.s2 + (static_cast<long long>(e) * NB + n0 / 128) * KB;      // 32 rows: one block of 128
    const int qlo = g < cnt ? pairs[g] : -1, qhi = g + 8 < cnt ? pairs[g + 8] : -1;
    const int elo = qlo >= 0 ? exponent_of(__ldcg(a.hmax + qlo)) : 0, ehi = qhi >= 0 ? exponent_of(__ldcg(a.hmax + qhi)) : 0;
    float out[kTiles][4];
#pragma unroll
    for (int i = 0; i < kTiles; ++i) out[i][0] = out[i][1] = out[i][2] = out[i][3] = 0.0f;
    for (int b = ba; b < bb; ++b) {
      const WBlock cur = next;
      if (b + 1 < bb) {
        load_wblock(next, row, (b + 1) * 128, F - t4 * 16);
      } else if (u_next < u1) {
        set_rows(u_next);
        load_wblock(next, row, u_next % KB * 128, F - t4 * 16);
      }
      const float s = __ldg(S + b);
      float blk[kTiles][4];
#pragma unroll
      for (int i = 0; i < kTiles; ++i) blk[i][0] = blk[i][1] = blk[i][2] = blk[i][3] = 0.0f;
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int k = b * 128 + c * 64 + t4 * 16;
        uint32_t lo[8], hi[8];
        load_hidden(lo, a, k < F ? qlo : -1, k, elo, strips);
        load_hidden(hi, a, k < F ? qhi : -1, k, ehi, strips);
        mma_run(blk, cur.w[c], lo, hi);
      }
#pragma unroll
      for (int i = 0; i < kTiles; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) out[i][j] = fmaf(blk[i][j], s, out[i][j]);
    }
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int q = half ? qhi : qlo;
      if (q < 0) continue;
      const float w = __ldcg(a.pair_w + q) * pow2((half ? ehi : elo) - 14);
      float* y = mine + q / KT * kPitch + 2 * t4;
#pragma unroll
      for (int i = 0; i < kTiles; ++i) {
        y[i * 8] = fmaf(w, out[i][half * 2], y[i * 8]);
        y[i * 8 + 1] = fmaf(w, out[i][half * 2 + 1], y[i * 8 + 1]);
      }
    }
    __syncwarp();
    p0 = more ? p0 + 16 : 0;
    u = u_next;
  }
  __syncthreads();
  if (a.split > 1) cluster_barrier();
  const uint32_t base = smem_u32(acc);
  for (int i = rank * kThreads + tid; i < T * kRows; i += a.split * kThreads) {
    const int t = i / kRows, r = i % kRows;
    float sum = 0.0f;
    for (int q = 0; q < a.split; ++q) {
      float v[kWarps];
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const uint32_t at = base + ((w * T + t) * kPitch + r) * 4;
        if (a.split > 1) asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v[w]) : "r"(mapa_u32(at, q)));
        else v[w] = acc[(w * T + t) * kPitch + r];
      }
#pragma unroll
      for (int w = 0; w < kWarps; ++w) sum += v[w];
    }
    if (n0 + r < D) a.y[static_cast<long long>(t) * D + n0 + r] = static_cast<uint16_t>(bf16x2_from_f32(sum, 0.0f));
  }
  if (a.split > 1) cluster_barrier();       // the others may still be reading this CTA's sums
}

size_t align256(size_t v) { return (v + 255) / 256 * 256; }

// Per device: shared-memory limits raised once.
constexpr int kMaxDevices = 64;
struct MoeSetup {
  std::once_flag once;
  cudaError_t err = cudaSuccess;
};
constexpr int kRouteSmemMax = 4 * BILOCO_MOE_MAX_D * 2, kDownSmemMax = kWarps * kMoeMaxTokens * (8 * kTiles + 1) * 4;

template <int kTok, bool kF32>
cudaError_t raise_route() {
  return cudaFuncSetAttribute(moe_route_kernel<kTok, kF32>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              kRouteSmemMax / 4 * kTok);
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
  take(a.hexp, P * (a.F / 16) * 4);
  take(a.xh, static_cast<size_t>(a.T) * a.D * 2);
  take(a.xscale, static_cast<size_t>(a.T) * 4);
  take(a.h, P * a.F * 2);
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
    const cudaError_t r[] = {raise_route<1, false>(), raise_route<1, true>(), raise_route<4, false>(),
                             raise_route<4, true>(),
                             cudaFuncSetAttribute(moe_down_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                  kDownSmemMax)};
    for (cudaError_t v : r)
      if (v != cudaSuccess) d.err = v;
  });
  if (d.err != cudaSuccess) return d.err;

  // up to 16 tokens a cluster each (128 CTAs); above, four tokens share a cluster's reads of the router
  const int tok = a.T <= 16 ? 1 : 4;
  const unsigned grid = static_cast<unsigned>((a.T + tok - 1) / tok * kRouteCtas);
  const size_t sm = static_cast<size_t>(tok) * a.D * 2;
  if (tok == 1)
    e = a.router_f32 ? launch_pdl(moe_route_kernel<1, true>, grid, kThreads, sm, kRouteCtas, s, a)
                     : launch_pdl(moe_route_kernel<1, false>, grid, kThreads, sm, kRouteCtas, s, a);
  else
    e = a.router_f32 ? launch_pdl(moe_route_kernel<4, true>, grid, kThreads, sm, kRouteCtas, s, a)
                     : launch_pdl(moe_route_kernel<4, false>, grid, kThreads, sm, kRouteCtas, s, a);
  if (e != cudaSuccess) return e;

  const int slots = 2 * num_sms();
  const int experts = min(a.T * a.k, a.E) + a.shared;
  const int items = experts * (a.F / 16);
  e = launch_pdl(moe_up_kernel, static_cast<unsigned>(min(slots, items)), kThreads, 0, 1, s, a);
  if (e != cudaSuccess) return e;

  // the cluster of an output strip is as large as one wave of CTAs allows
  const int rows = (a.D + 8 * kTiles - 1) / (8 * kTiles);
  a.split = max(1, min(8, slots / rows));
  return launch_pdl(moe_down_kernel, static_cast<unsigned>(rows * a.split), kThreads,
                    static_cast<size_t>(kWarps) * a.T * (8 * kTiles + 1) * 4, static_cast<unsigned>(a.split), s, a);
}

}  // namespace biloco
