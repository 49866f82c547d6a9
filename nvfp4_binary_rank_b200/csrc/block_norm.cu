// The step between two blocks of a transformer layer in one pass: the norm after a
// block, its gate, the scaled residual sum, and the norm before the next block.
//
//   u  = y * rsqrt(mean(y^2) + eps) * (post_w + offset)        (u = y without post_w)
//   h' = res_scale * h + gate * u
//   x  = h' * rsqrt(mean(h'^2) + eps) * (pre_w + offset)       (BF16, or FP8 blocks)
//
// Bound by memory: y and h are read once, h' and x written once, and the row stays in
// registers between the two norms.  A CTA takes a row at a time, a thread kVec pieces of eight
// elements.  CTAs stay: each walks over rows with the loads of its next row under way while
// the current one goes through its two sums.  y and h pass by L1, which so keeps the weights.
// Measured at 8192 x 5120 with FP8 output (295 MB): one CTA per row 85 us, this NEW us.
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

// Eight consecutive values as they lie in memory (BF16 or FP32), and widened.
template <bool kF32>
struct Raw8 {
  uint4 q[kF32 ? 2 : 1];
  // weights and gates: cached
  __device__ __forceinline__ void load(const void* p, long long at) {
    const uint4* s = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(p) + at * (kF32 ? 4 : 2));
    q[0] = __ldg(s);
    if (kF32) q[kF32] = __ldg(s + 1);
  }
  // rows: read once, and perhaps written by this kernel (h' over h)
  __device__ __forceinline__ void stream(const void* p, long long at) {
    const uint8_t* s = static_cast<const uint8_t*>(p) + at * (kF32 ? 4 : 2);
    take(q[0], s);
    if (kF32) take(q[kF32], s + 16);
  }
  static __device__ __forceinline__ void take(uint4& v, const uint8_t* p) {
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p) : "memory");
  }
  __device__ __forceinline__ void zero() {
    q[0] = make_uint4(0, 0, 0, 0);
    if (kF32) q[kF32] = make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ float at(int j) const {
    if (kF32) {
      const uint4& v = q[kF32 ? j >> 2 : 0];
      return __uint_as_float((j & 3) == 0 ? v.x : (j & 3) == 1 ? v.y : (j & 3) == 2 ? v.z : v.w);
    }
    const uint32_t w = (j >> 1) == 0 ? q[0].x : (j >> 1) == 1 ? q[0].y : (j >> 1) == 2 ? q[0].z : q[0].w;
    return (j & 1) ? bf16_hi(w) : bf16_lo(w);
  }
};

__device__ __forceinline__ uint4 to_bf16x8(const float (&v)[8]) {
  return make_uint4(bf16x2_from_f32(v[0], v[1]), bf16x2_from_f32(v[2], v[3]), bf16x2_from_f32(v[4], v[5]),
                    bf16x2_from_f32(v[6], v[7]));
}

// Sum over the CTA; every thread gets it, summed in the same order.  `part` has one slot per
// warp; its next use is a barrier later (the row's other sum, or the next row's).
__device__ __forceinline__ float cta_sum(float v, float* part) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  const int warps = blockDim.x >> 5, lane = threadIdx.x & 31;
  if (warps == 1) return v;
  if (lane == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  v = lane < warps ? part[lane] : 0.0f;
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

template <int kVec, int kMaxThreads, bool kAhead, bool kHf32, bool kWf32>
__global__ void __launch_bounds__(kMaxThreads, kMaxThreads == 512 && !kHf32 ? 2 : 1)
block_norm_kernel(const __grid_constant__ BlockNormArgs a) {
  __shared__ float part[2][32];
  const int D = a.D, nvec = D >> 3, step = static_cast<int>(gridDim.x);
  auto piece = [&](int i) { return static_cast<int>(threadIdx.x + i * blockDim.x); };
  struct Row {
    Raw8<false> y[kVec];
    Raw8<kHf32> h[kVec];
  };
  auto load_row = [&](Row& r, int m) {
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      r.y[i].zero();
      r.h[i].zero();
      if (piece(i) < nvec) {
        if (a.y) r.y[i].stream(a.y, m * a.ldy + piece(i) * 8);
        if (a.h) r.h[i].stream(a.h, m * a.ldh + piece(i) * 8);
      }
    }
  };
  griddep_launch_dependents();
  griddep_wait();
  Row next;
  if (kAhead) load_row(next, static_cast<int>(blockIdx.x));
  for (int m = static_cast<int>(blockIdx.x); m < a.M; m += step) {
    Row row;
    if (kAhead) {
      row = next;
      if (m + step < a.M) load_row(next, m + step);
    } else {
      load_row(row, m);
    }
    float post = 1.0f;
    if (a.post_w) {
      float ss = 0.0f;
#pragma unroll
      for (int i = 0; i < kVec; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) ss = fmaf(row.y[i].at(j), row.y[i].at(j), ss);
      post = rsqrtf(cta_sum(ss, part[0]) / static_cast<float>(D) + a.eps);
    }
    const long long gate_at = static_cast<long long>(a.gate ? m / a.rows_per_gate : 0) * D;
    float r[kVec][8];
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      if (piece(i) >= nvec) continue;
#pragma unroll
      for (int j = 0; j < 8; ++j) r[i][j] = row.y[i].at(j);
      if (a.post_w) {
        Raw8<kWf32> w;
        w.load(a.post_w, piece(i) * 8);
#pragma unroll
        for (int j = 0; j < 8; ++j) r[i][j] = r[i][j] * post * (w.at(j) + a.offset);
      }
      if (a.gate && a.gate_f32) {
        Raw8<true> g;
        g.load(a.gate, gate_at + piece(i) * 8);
#pragma unroll
        for (int j = 0; j < 8; ++j) r[i][j] *= g.at(j);
      } else if (a.gate) {
        Raw8<false> g;
        g.load(a.gate, gate_at + piece(i) * 8);
#pragma unroll
        for (int j = 0; j < 8; ++j) r[i][j] *= g.at(j);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        r[i][j] = fmaf(a.res_scale, row.h[i].at(j), r[i][j]);
        ss = fmaf(r[i][j], r[i][j], ss);
      }
      if (a.h_out) {
        const long long at = m * a.ldho + piece(i) * 8;
        if (kHf32) {
          float4* q = reinterpret_cast<float4*>(static_cast<float*>(a.h_out) + at);
          q[0] = make_float4(r[i][0], r[i][1], r[i][2], r[i][3]);
          q[1] = make_float4(r[i][4], r[i][5], r[i][6], r[i][7]);
        } else {
          *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.h_out) + at) = to_bf16x8(r[i]);
        }
      }
    }
    if (!a.pre_w) {
      if (a.post_w) __syncthreads();      // the one sum of this row is read before the next row's is written
      continue;
    }
    const float s = rsqrtf(cta_sum(ss, part[1]) / static_cast<float>(D) + a.eps);
    uint32_t top[kVec];
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      const int c = piece(i);
      top[i] = 0;
      if (c < nvec) {
        Raw8<kWf32> w;
        w.load(a.pre_w, c * 8);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          r[i][j] = r[i][j] * s * (w.at(j) + a.offset);
          top[i] = max(top[i], __float_as_uint(r[i][j]) & 0x7FFFFFFFu);
        }
        if (a.x_out) *reinterpret_cast<uint4*>(a.x_out + static_cast<long long>(m) * D + c * 8) = to_bf16x8(r[i]);
      }
    }
    if (a.codes) {
      // 16 lanes hold a block of 128 (a piece index is a multiple of 16 at every 16th lane);
      // lane i of the 16 does the two divisions of piece i's block
      const int who = threadIdx.x & 15;
      uint32_t mine = 0;
#pragma unroll
      for (int i = 0; i < kVec; ++i) {
#pragma unroll
        for (int o = 8; o; o >>= 1) top[i] = max(top[i], __shfl_xor_sync(0xFFFFFFFFu, top[i], o));
        if (who == i) mine = top[i];
      }
      const Fp8Scale f = fp8_block_scale(mine);
#pragma unroll
      for (int i = 0; i < kVec; ++i) {
        const int c = piece(i);
        const float inv = __shfl_sync(0xFFFFFFFFu, f.inv, i, 16);
        if (c >= nvec) continue;
        *reinterpret_cast<uint2*>(a.codes + static_cast<long long>(m) * D + c * 8) =
            make_uint2(e4m3x4_from_f32(__fmul_rn(r[i][0], inv), __fmul_rn(r[i][1], inv), __fmul_rn(r[i][2], inv),
                                       __fmul_rn(r[i][3], inv)),
                       e4m3x4_from_f32(__fmul_rn(r[i][4], inv), __fmul_rn(r[i][5], inv), __fmul_rn(r[i][6], inv),
                                       __fmul_rn(r[i][7], inv)));
      }
      // lane i also stores that block's scale; its own piece i may lie past the row's end when the block does not
#pragma unroll
      for (int i = 0; i < kVec; ++i) {
        const int blk = piece(i) >> 4;
        if (who == i && blk < (D + 127) / 128) a.scales[static_cast<size_t>(blk) * a.M + m] = f.scale;
      }
    }
    // With one sum per row, and a single barrier in it, a fast warp could write the next row's
    // part while a slow one still reads this row's.
    if (!a.post_w) __syncthreads();
  }
}

template <int kVec, int kMaxThreads, bool kAhead, bool kHf32, bool kWf32>
cudaError_t launch_one(const BlockNormArgs& a, cudaStream_t s) {
  auto kernel = block_norm_kernel<kVec, kMaxThreads, kAhead, kHf32, kWf32>;
  const int nvec = a.D / 8, warps = ((nvec + kVec - 1) / kVec + 31) / 32;
  // as many CTAs as run at once, at most one per row
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
  // A few rows: one piece a thread, the shortest way through a row.  Many: two, so that
  // several rows are under way on an SM (four with half the threads: 5% slower).  Above 8192
  // columns the registers do not hold a second row.
  if (a.D <= 2048 || (a.D <= 8192 && a.M <= num_sms())) return launch_one<1, 1024, true, kHf32, kWf32>(a, s);
  if (a.D <= 8192) return launch_one<2, 512, true, kHf32, kWf32>(a, s);
  return launch_one<4, 1024, false, kHf32, kWf32>(a, s);
}

}  // namespace

cudaError_t launch_block_norm(const BlockNormArgs& a, cudaStream_t s) {
  if (a.h_f32) return a.w_f32 ? launch_typed<true, true>(a, s) : launch_typed<true, false>(a, s);
  return a.w_f32 ? launch_typed<false, true>(a, s) : launch_typed<false, false>(a, s);
}

}  // namespace biloco
