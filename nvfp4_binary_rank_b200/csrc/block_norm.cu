// The step between two blocks of a transformer layer in one pass: the norm after a
// block, its gate, the scaled residual sum, and the norm before the next block.
//
//   u  = y * rsqrt(mean(y^2) + eps) * (post_w + offset)        (u = y without post_w)
//   h' = res_scale * h + gate * u
//   x  = h' * rsqrt(mean(h'^2) + eps) * (pre_w + offset)       (BF16, or FP8 blocks)
//
// Bound by memory: y and h are read once, h' and x written once, and the row stays in
// registers between the two norms.  A CTA takes a row at a time, a thread kVec pieces of eight
// elements, two at a time in packed FP32 arithmetic (with single operations the kernel issued
// 696 instructions a warp and row and was bound by them).  CTAs stay: each walks over rows,
// and the loads of its next row are under way from the middle of the current one, when the
// registers of that are free.  y and h pass by L1, which so keeps the weights.
// Measured at 8192 x 5120 with FP8 output (295 MB): one CTA per row 85 us, this 63 to 66 us (4.5 TB/s,
// instructions issued in 65% of the clocks); with BF16 output (336 MB) 61 us, 5.5 TB/s.  Neither
// memory nor the issue slots are full: a row waits for two sums over its CTA, and three rows
// are under way on an SM.  One row of 5120 takes 2.5 to 3.0 us, the two sums and the loads before them.
// Rows above 8192 (four pieces a thread, one CTA of 1024 an SM at 64 registers, 200 to 372 bytes of
// them spilled): 2048 x 16384 in 76 us with FP8 and 69 us with BF16 output, 1024 x 32768 in 82 and 75
// (floors 36 and 41).
// Both sums of squares are FP32; x is computed from the unrounded h', so h' and x are each
// rounded once.
#include <algorithm>
#include <atomic>
#include <cstdint>

#include <cuda_runtime.h>

#include "fp8_dev.cuh"
#include "fp8_ops.h"
#include "internal.h"
#include "ptx.cuh"

namespace biloco {

namespace {

// Eight consecutive values as they lie in memory (BF16 or FP32), widened in pairs.
template <bool kF32>
struct Raw8 {
  uint4 q[kF32 ? 2 : 1];
  // weights and gates: cached
  __device__ __forceinline__ void load(const void* p, int at) {
    const uint4* s = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(p) + at * (kF32 ? 4 : 2));
    q[0] = __ldg(s);
    if (kF32) q[kF32] = __ldg(s + 1);
  }
  // rows: read once, and perhaps written by this kernel (h' over h)
  __device__ __forceinline__ void stream(const uint8_t* p) {
    take(q[0], p);
    if (kF32) take(q[kF32], p + 16);
  }
  static __device__ __forceinline__ void take(uint4& v, const uint8_t* p) {
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p) : "memory");
  }
  __device__ __forceinline__ void zero() {
    q[0] = make_uint4(0, 0, 0, 0);
    if (kF32) q[kF32] = make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ uint64_t pair(int j) const {          // values 2 j and 2 j + 1
    if (kF32) {
      const uint4& v = q[kF32 ? j >> 1 : 0];
      return (j & 1) ? f32x2_pack(v.z, v.w) : f32x2_pack(v.x, v.y);
    }
    const uint32_t w = j == 0 ? q[0].x : j == 1 ? q[0].y : j == 2 ? q[0].z : q[0].w;
    return f32x2_pack(w << 16, w & 0xFFFF0000u);
  }
};

__device__ __forceinline__ uint64_t f32x2_mul(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t f32x2_add(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t both(float v) { return f32x2_pack(__float_as_uint(v), __float_as_uint(v)); }
__device__ __forceinline__ void split(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint32_t pack_bf16(uint64_t v) {
  float lo, hi;
  split(v, lo, hi);
  return bf16x2_from_f32(lo, hi);
}
// max(a, |lo|, |hi|), NaN if any is
__device__ __forceinline__ float max_abs(float a, uint64_t v) {
  float lo, hi;
  split(v, lo, hi);
  asm("max.NaN.f32 %0, %0, %1;" : "+f"(a) : "f"(fabsf(lo)));
  asm("max.NaN.f32 %0, %0, %1;" : "+f"(a) : "f"(fabsf(hi)));
  return a;
}

// Sum over the CTA; every thread gets it, summed in the same order.  `part` has one slot per
// warp, zeros behind them; its next use is a barrier later (the row's other sum, or the next row's).
// Each thread adds up the slots itself: reads of shared memory at once, where shuffles
// would be five dependent steps.
template <int kSlots>
__device__ __forceinline__ float cta_sum(float v, float4* part) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  const int warps = blockDim.x >> 5, lane = threadIdx.x & 31;
  if (warps == 1) return v;
  if (lane == 0) reinterpret_cast<float*>(part)[threadIdx.x >> 5] = v;
  __syncthreads();
  float4 s = part[0];
#pragma unroll
  for (int i = 1; i < kSlots / 4; ++i) {
    if (4 * i >= warps) break;
    const float4 q = part[i];
    s.x += q.x;
    s.y += q.y;
    s.z += q.z;
    s.w += q.w;
  }
  return (s.x + s.y) + (s.z + s.w);
}

template <int kVec, int kMaxThreads, bool kHf32, bool kWf32>
__global__ void __launch_bounds__(kMaxThreads, kMaxThreads == 512 ? 2 : 1)
block_norm_kernel(const __grid_constant__ BlockNormArgs a) {
  constexpr int kSlots = kMaxThreads / 32;
  __shared__ float4 part[2][kSlots / 4];
  const int D = a.D, nvec = D >> 3;
  constexpr int kHb = kHf32 ? 4 : 2;
  int at[kVec];                                // first element of this thread's pieces
  bool in[kVec];
  Raw8<false> y[kVec];
  Raw8<kHf32> h[kVec];
#pragma unroll
  for (int i = 0; i < kVec; ++i) {
    const int c = static_cast<int>(threadIdx.x + i * blockDim.x);
    in[i] = c < nvec;
    at[i] = c * 8;
    y[i].zero();                               // pieces past the row's end stay zero
    h[i].zero();
  }
  auto load_row = [&](int m) {
    const uint8_t* py = reinterpret_cast<const uint8_t*>(a.y) + m * a.ldy * 2;
    const uint8_t* ph = static_cast<const uint8_t*>(a.h) + m * a.ldh * kHb;
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      if (in[i] && a.y) y[i].stream(py + at[i] * 2);
      if (in[i] && a.h) h[i].stream(ph + at[i] * kHb);
    }
  };
  griddep_launch_dependents();
  if (threadIdx.x < 2 * kSlots) reinterpret_cast<float*>(part)[threadIdx.x] = 0.0f;
  __syncthreads();
  griddep_wait();
  load_row(static_cast<int>(blockIdx.x));
  const float inv_d = 1.0f / static_cast<float>(D);
  const uint64_t offset = both(a.offset), res = both(a.res_scale);
#pragma unroll 1
  for (int m = static_cast<int>(blockIdx.x); m < a.M; m += static_cast<int>(gridDim.x)) {
    uint64_t post = both(1.0f);
    if (a.post_w) {
      uint64_t ss = 0;
#pragma unroll
      for (int i = 0; i < kVec; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint64_t v = y[i].pair(j);
          ss = f32x2_fma(v, v, ss);
        }
      post = both(rsqrtf(cta_sum<kSlots>(f32x2_sum(ss), part[0]) * inv_d + a.eps));
    }
    uint64_t r[kVec][4], ss = 0;
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
#pragma unroll
      for (int j = 0; j < 4; ++j) r[i][j] = y[i].pair(j);
      if (!in[i]) continue;
      if (a.post_w) {
        Raw8<kWf32> w;
        w.load(a.post_w, at[i]);
#pragma unroll
        for (int j = 0; j < 4; ++j) r[i][j] = f32x2_mul(f32x2_mul(r[i][j], post), f32x2_add(w.pair(j), offset));
      }
      if (a.gate) {
        const uint8_t* g = static_cast<const uint8_t*>(a.gate) +
                           static_cast<long long>(m / a.rows_per_gate) * D * (a.gate_f32 ? 4 : 2);
        if (a.gate_f32) {
          Raw8<true> v;
          v.load(g, at[i]);
#pragma unroll
          for (int j = 0; j < 4; ++j) r[i][j] = f32x2_mul(r[i][j], v.pair(j));
        } else {
          Raw8<false> v;
          v.load(g, at[i]);
#pragma unroll
          for (int j = 0; j < 4; ++j) r[i][j] = f32x2_mul(r[i][j], v.pair(j));
        }
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        r[i][j] = f32x2_fma(res, h[i].pair(j), r[i][j]);
        ss = f32x2_fma(r[i][j], r[i][j], ss);
      }
      if (a.h_out) {
        uint8_t* p = static_cast<uint8_t*>(a.h_out) + (m * a.ldho + at[i]) * kHb;
        if (kHf32) {
          ulonglong2* q = reinterpret_cast<ulonglong2*>(p);
          q[0] = make_ulonglong2(r[i][0], r[i][1]);
          q[1] = make_ulonglong2(r[i][2], r[i][3]);
        } else {
          *reinterpret_cast<uint4*>(p) =
              make_uint4(pack_bf16(r[i][0]), pack_bf16(r[i][1]), pack_bf16(r[i][2]), pack_bf16(r[i][3]));
        }
      }
    }
    if (m + static_cast<int>(gridDim.x) < a.M) load_row(m + static_cast<int>(gridDim.x));
    if (!a.pre_w) {
      if (a.post_w) __syncthreads();      // the one sum of this row is read before the next row's is written
      continue;
    }
    const uint64_t pre = both(rsqrtf(cta_sum<kSlots>(f32x2_sum(ss), part[1]) * inv_d + a.eps));
    float top[kVec];
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      top[i] = 0.0f;
      if (!in[i]) continue;
      Raw8<kWf32> w;
      w.load(a.pre_w, at[i]);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        r[i][j] = f32x2_mul(f32x2_mul(r[i][j], pre), f32x2_add(w.pair(j), offset));
        if (a.codes) top[i] = max_abs(top[i], r[i][j]);
      }
      if (a.x_out)
        *reinterpret_cast<uint4*>(a.x_out + static_cast<long long>(m) * D + at[i]) =
            make_uint4(pack_bf16(r[i][0]), pack_bf16(r[i][1]), pack_bf16(r[i][2]), pack_bf16(r[i][3]));
    }
    if (a.codes) {
      // 16 lanes hold a block of 128 (a piece index is a multiple of 16 at every 16th lane);
      // lane i of the 16 does the two divisions of piece i's block and stores its scale
      const int who = threadIdx.x & 15;
      uint32_t mine = 0;
#pragma unroll
      for (int i = 0; i < kVec; ++i) {
        uint32_t t = __float_as_uint(top[i]);        // not negative, NaN above all: ordered as integers
#pragma unroll
        for (int o = 8; o; o >>= 1) t = max(t, __shfl_xor_sync(0xFFFFFFFFu, t, o));
        if (who == i) mine = t;
      }
      const Fp8Scale f = fp8_block_scale(mine & 0x7FFFFFFFu);
#pragma unroll
      for (int i = 0; i < kVec; ++i) {
        const uint64_t inv = both(__shfl_sync(0xFFFFFFFFu, f.inv, i, 16));
        const int blk = at[i] >> 7;
        if (who == i && blk < (D + 127) / 128) a.scales[static_cast<size_t>(blk) * a.M + m] = f.scale;
        if (!in[i]) continue;
        float v[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) split(f32x2_mul(r[i][j], inv), v[2 * j], v[2 * j + 1]);
        *reinterpret_cast<uint2*>(a.codes + static_cast<long long>(m) * D + at[i]) =
            make_uint2(e4m3x4_from_f32(v[0], v[1], v[2], v[3]), e4m3x4_from_f32(v[4], v[5], v[6], v[7]));
      }
    }
    // With one sum per row, and a single barrier in it, a fast warp could write the next row's
    // part while a slow one still reads this row's.
    if (!a.post_w) __syncthreads();
  }
}

template <int kVec, int kMaxThreads, bool kHf32, bool kWf32>
cudaError_t launch_one(const BlockNormArgs& a, cudaStream_t s) {
  auto kernel = block_norm_kernel<kVec, kMaxThreads, kHf32, kWf32>;
  const int nvec = a.D / 8, warps = ((nvec + kVec - 1) / kVec + 31) / 32;
  // as many CTAs as run at once, at most one per row; every GPU this library takes holds as many an SM
  static std::atomic<int> per_sm[kMaxThreads / 32 + 1];
  int n = per_sm[warps].load();
  if (n == 0) {
    const cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, warps * 32, 0);
    if (e != cudaSuccess) return e;
    per_sm[warps].store(n = std::max(n, 1));
  }
  const unsigned grid = static_cast<unsigned>(std::min(a.M, n * num_sms()));
  return launch_pdl(kernel, grid, static_cast<unsigned>(warps * 32), 0, 1, s, a);
}

template <bool kHf32, bool kWf32>
cudaError_t launch_typed(const BlockNormArgs& a, cudaStream_t s) {
  // Short rows, and as many as one round of CTAs takes: one piece a thread, the shortest way
  // through a row.  More: two, so that several rows are under way on an SM.  Four where two
  // need more than 512 threads.  Measured with FP8 output, us with one and two pieces: 2.6 and 3.1
  // (1 x 5120), 3.4 and 4.0 (148 x 5120), 4.6 and 4.3 (149 x 5120), 92 and 65 (8192 x 5120); 3.6 and
  // 4.1 (592 x 2048), 27.4 and 24.5 (8192 x 2048); 14.5 and 14.4 (8192 x 1024), 8.0 and 9.0
  // (8192 x 512).  Four pieces: 94 (8192 x 5120).
  const int threads = (a.D / 8 + 31) / 32 * 32;
  if (a.D <= 1024 || (threads <= 1024 && a.M <= 1024 / threads * num_sms())) return launch_one<1, 1024, kHf32, kWf32>(a, s);
  if (a.D <= 8192) return launch_one<2, 512, kHf32, kWf32>(a, s);
  return launch_one<4, 1024, kHf32, kWf32>(a, s);
}

}  // namespace

cudaError_t launch_block_norm(const BlockNormArgs& a, cudaStream_t s) {
  if (a.h_f32) return a.w_f32 ? launch_typed<true, true>(a, s) : launch_typed<true, false>(a, s);
  return a.w_f32 ? launch_typed<false, true>(a, s) : launch_typed<false, false>(a, s);
}

}  // namespace biloco
