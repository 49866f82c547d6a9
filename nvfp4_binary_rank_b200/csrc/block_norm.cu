// The step between two blocks of a transformer layer in one pass: the norm after a
// block, its gate, the scaled residual sum, and the norm before the next block.
//
//   u  = y * rsqrt(mean(y^2) + eps) * (post_w + offset)        (u = y without post_w)
//   h' = res_scale * h + gate * u
//   x  = h' * rsqrt(mean(h'^2) + eps) * (pre_w + offset)       (BF16, or FP8 blocks)
//
// Bound by memory: y and h are read once, h' and x written once, and the row stays in
// registers between the two norms.  One CTA per row; a thread owns kVec pieces of eight
// elements (16 bytes of BF16).  Both sums of squares are FP32; x is computed from the
// unrounded h', so h' and x are each rounded once.
#include <cstdint>
#include <cuda_runtime.h>

#include "fp8_dev.cuh"
#include "fp8_ops.h"
#include "internal.h"
#include "ptx.cuh"

namespace biloco {

namespace {

// Eight consecutive values at element offset `at` of an array of BF16 or FP32.
__device__ __forceinline__ void load8(const void* p, bool f32, long long at, float (&v)[8]) {
  if (f32) {
    const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(p) + at);
    const float4 a = q[0], b = q[1];
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  } else {
    const uint4 a = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + at);
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[2 * j] = bf16_lo(w[j]);
      v[2 * j + 1] = bf16_hi(w[j]);
    }
  }
}

__device__ __forceinline__ uint4 to_bf16x8(const float (&v)[8]) {
  return make_uint4(bf16x2_from_f32(v[0], v[1]), bf16x2_from_f32(v[2], v[3]), bf16x2_from_f32(v[4], v[5]),
                    bf16x2_from_f32(v[6], v[7]));
}

// Sum over the CTA; every thread gets it, summed in the same order.  `part` has one
// slot per warp and is used once per row, so one barrier is enough.
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

template <int kVec, bool kHf32>
__global__ void __launch_bounds__(256 * kVec)
block_norm_kernel(const __grid_constant__ BlockNormArgs a) {
  griddep_launch_dependents();
  griddep_wait();
  __shared__ float part[2][32];
  const int D = a.D, nvec = D >> 3;
  const long long m = blockIdx.x;
  float u[kVec][8], h[kVec][8];
#pragma unroll
  for (int i = 0; i < kVec; ++i) {
    const int c = threadIdx.x + i * blockDim.x;
#pragma unroll
    for (int j = 0; j < 8; ++j) u[i][j] = h[i][j] = 0.0f;
    if (c < nvec) {
      if (a.y) load8(a.y, false, m * a.ldy + c * 8, u[i]);
      if (a.h) load8(a.h, kHf32, m * a.ldh + c * 8, h[i]);
    }
  }
  if (a.post_w) {
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < kVec; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) ss = fmaf(u[i][j], u[i][j], ss);
    const float r = rsqrtf(cta_sum(ss, part[0]) / static_cast<float>(D) + a.eps);
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      const int c = threadIdx.x + i * blockDim.x;
      if (c < nvec) {
        float w[8];
        load8(a.post_w, a.w_f32, c * 8, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) u[i][j] = u[i][j] * r * (w[j] + a.offset);
      }
    }
  }
  float ss = 0.0f;
#pragma unroll
  for (int i = 0; i < kVec; ++i) {
    const int c = threadIdx.x + i * blockDim.x;
    if (c < nvec) {
      if (a.gate) {
        float g[8];
        load8(a.gate, a.gate_f32, (m / a.rows_per_gate) * D + c * 8, g);
#pragma unroll
        for (int j = 0; j < 8; ++j) u[i][j] *= g[j];
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        h[i][j] = fmaf(a.res_scale, h[i][j], u[i][j]);
        ss = fmaf(h[i][j], h[i][j], ss);
      }
      if (a.h_out) {
        const long long at = m * a.ldho + c * 8;
        if (kHf32) {
          float4* q = reinterpret_cast<float4*>(static_cast<float*>(a.h_out) + at);
          q[0] = make_float4(h[i][0], h[i][1], h[i][2], h[i][3]);
          q[1] = make_float4(h[i][4], h[i][5], h[i][6], h[i][7]);
        } else {
          *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.h_out) + at) = to_bf16x8(h[i]);
        }
      }
    }
  }
  if (!a.pre_w) return;
  const float r = rsqrtf(cta_sum(ss, part[1]) / static_cast<float>(D) + a.eps);
#pragma unroll
  for (int i = 0; i < kVec; ++i) {
    const int c = threadIdx.x + i * blockDim.x;
    const bool in = c < nvec;
    uint32_t top = 0;
    if (in) {
      float w[8];
      load8(a.pre_w, a.w_f32, c * 8, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        h[i][j] = h[i][j] * r * (w[j] + a.offset);
        top = max(top, __float_as_uint(h[i][j]) & 0x7FFFFFFFu);
      }
      if (a.x_out) *reinterpret_cast<uint4*>(a.x_out + m * D + c * 8) = to_bf16x8(h[i]);
    }
    if (a.codes) {
      // 16 lanes hold a block of 128: c is a multiple of 16 at every 16th lane
#pragma unroll
      for (int o = 8; o; o >>= 1) top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
      const Fp8Scale s = fp8_block_scale(top);
      if (in) {
        *reinterpret_cast<uint2*>(a.codes + m * D + c * 8) =
            make_uint2(e4m3x4_from_f32(__fmul_rn(h[i][0], s.inv), __fmul_rn(h[i][1], s.inv),
                                       __fmul_rn(h[i][2], s.inv), __fmul_rn(h[i][3], s.inv)),
                       e4m3x4_from_f32(__fmul_rn(h[i][4], s.inv), __fmul_rn(h[i][5], s.inv),
                                       __fmul_rn(h[i][6], s.inv), __fmul_rn(h[i][7], s.inv)));
        if ((threadIdx.x & 15) == 0) a.scales[static_cast<size_t>(c >> 4) * a.M + m] = s.scale;
      }
    }
  }
}

template <int kVec>
cudaError_t launch_vec(const BlockNormArgs& a, unsigned threads, cudaStream_t s) {
  return a.h_f32 ? launch_pdl(block_norm_kernel<kVec, true>, static_cast<unsigned>(a.M), threads, 0, 1, s, a)
                 : launch_pdl(block_norm_kernel<kVec, false>, static_cast<unsigned>(a.M), threads, 0, 1, s, a);
}

}  // namespace

cudaError_t launch_block_norm(const BlockNormArgs& a, cudaStream_t s) {
  const int nvec = a.D / 8;
  const int vec = nvec <= 256 ? 1 : nvec <= 1024 ? 2 : 4;
  const unsigned threads = static_cast<unsigned>(((nvec + vec - 1) / vec + 31) / 32 * 32);
  if (vec == 1) return launch_vec<1>(a, threads, s);
  if (vec == 2) return launch_vec<2>(a, threads, s);
  return launch_vec<4>(a, threads, s);
}

}  // namespace biloco
