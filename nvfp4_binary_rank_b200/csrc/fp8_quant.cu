// FP8 block quantisers: activations per 128 elements of a row, weights per 128 x 128
// tile (the format is in fp8_dev.cuh).  Both are one pass over the data.
#include <cstdint>
#include <cuda_runtime.h>

#include "fp8_dev.cuh"
#include "fp8_ops.h"
#include "ptx.cuh"

namespace biloco {

namespace {

constexpr int kThreads = 256;

// One lane holds 16 elements (two 16-byte loads, one 16-byte store), so eight lanes
// hold a block and its maximum is three shuffles.  A warp covers 512 elements of a row.
// Bound by memory: 8192 x 5120 (127 MB) in 21.0 us past L2, 6.1 TB/s; 32 x 13824 takes 1.7 us, the
// time of one kernel in a row of them.
__global__ void __launch_bounds__(kThreads)
fp8_quant_act_kernel(const uint16_t* __restrict__ x, long long ldx, int M, int K, int chunks,
                     uint8_t* __restrict__ codes, float* __restrict__ scales) {
  griddep_launch_dependents();
  griddep_wait();
  const long long wid = (static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x) >> 5;
  const int lane = threadIdx.x & 31;
  const long long m = wid / chunks;
  if (m >= M) return;                                   // whole warp leaves together
  const int k = static_cast<int>(wid % chunks) * 512 + lane * 16;
  const bool in = k < K;                                // K % 16 == 0: a lane is whole or absent
  uint4 a = make_uint4(0, 0, 0, 0), b = a;
  if (in) {
    const uint4* p = reinterpret_cast<const uint4*>(x + m * ldx + k);
    a = __ldg(p);
    b = __ldg(p + 1);
  }
  const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  uint32_t top = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) top = __vmaxu2(top, w[j] & 0x7FFF7FFFu);
  top = max(top << 16, top & 0xFFFF0000u);
#pragma unroll
  for (int o = 4; o; o >>= 1) top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
  const Fp8Scale s = fp8_block_scale(top);
  if (!in) return;
  uint32_t c[4];
#pragma unroll
  for (int j = 0; j < 4; ++j)
    c[j] = e4m3x4_from_f32(__fmul_rn(bf16_lo(w[2 * j]), s.inv), __fmul_rn(bf16_hi(w[2 * j]), s.inv),
                           __fmul_rn(bf16_lo(w[2 * j + 1]), s.inv), __fmul_rn(bf16_hi(w[2 * j + 1]), s.inv));
  *reinterpret_cast<uint4*>(codes + m * K + k) = make_uint4(c[0], c[1], c[2], c[3]);
  if ((lane & 7) == 0) scales[static_cast<size_t>(k / kFp8Block) * M + m] = s.scale;
}

// Bound by memory: 13824 x 5120 from BF16 in 34.8 us (6.1 TB/s), from FP32 in 56.3 us (6.3 TB/s);
// 5120 x 5120 in 12.8 and 23.0 us.
// One CTA per 128 x 128 tile: a thread keeps four 16-element pieces in registers
// (eight threads across a row, 32 rows apart), so the tile is read once.
template <bool kF32>
__global__ void __launch_bounds__(kThreads)
fp8_pack_weight_kernel(const void* __restrict__ W, int N, int K, int NB, int KB,
                       uint8_t* __restrict__ codes, float* __restrict__ scales) {
  const int kb = blockIdx.x % KB;
  const int nb = blockIdx.x / KB % NB;
  const long long row0 = static_cast<long long>(blockIdx.x / KB / NB) * N;    // expert's first row
  const int t = threadIdx.x;
  const int k = kb * kFp8Block + (t & 7) * 16;
  float v[4][16];
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int n = nb * kFp8Block + i * 32 + (t >> 3);
    const bool in = n < N && k < K;
    if (kF32) {
      const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(W) + (row0 + n) * K + k);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float4 q = in ? __ldg(p + j) : make_float4(0, 0, 0, 0);
        v[i][4 * j] = q.x; v[i][4 * j + 1] = q.y; v[i][4 * j + 2] = q.z; v[i][4 * j + 3] = q.w;
      }
    } else {
      const uint4* p = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(W) + (row0 + n) * K + k);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const uint4 q = in ? __ldg(p + j) : make_uint4(0, 0, 0, 0);
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          v[i][8 * j + 2 * u] = bf16_lo(w[u]);
          v[i][8 * j + 2 * u + 1] = bf16_hi(w[u]);
        }
      }
    }
#pragma unroll
    for (int j = 0; j < 16; ++j) top = max(top, __float_as_uint(v[i][j]) & 0x7FFFFFFFu);
  }
  __shared__ uint32_t part[kThreads / 32];
#pragma unroll
  for (int o = 16; o; o >>= 1) top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
  if ((t & 31) == 0) part[t >> 5] = top;
  __syncthreads();
#pragma unroll
  for (int j = 0; j < kThreads / 32; ++j) top = max(top, part[j]);
  const Fp8Scale s = fp8_block_scale(top);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int n = nb * kFp8Block + i * 32 + (t >> 3);
    if (n >= N || k >= K) continue;
    uint32_t c[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      c[j] = e4m3x4_from_f32(__fmul_rn(v[i][4 * j], s.inv), __fmul_rn(v[i][4 * j + 1], s.inv),
                             __fmul_rn(v[i][4 * j + 2], s.inv), __fmul_rn(v[i][4 * j + 3], s.inv));
    *reinterpret_cast<uint4*>(codes + (row0 + n) * K + k) = make_uint4(c[0], c[1], c[2], c[3]);
  }
  if (t == 0) scales[blockIdx.x] = s.scale;
}

}  // namespace

cudaError_t launch_fp8_quant_act(const uint16_t* x, long long ldx, int M, int K, uint8_t* codes, float* scales,
                                 cudaStream_t s) {
  const int chunks = (K + 511) / 512;
  const long long warps = static_cast<long long>(M) * chunks;
  const long long grid = (warps + kThreads / 32 - 1) / (kThreads / 32);
  if (grid > 0x7FFFFFFFLL) return cudaErrorInvalidConfiguration;
  return launch_pdl(fp8_quant_act_kernel, static_cast<unsigned>(grid), kThreads, 0, 1, s, x, ldx, M, K, chunks, codes,
                    scales);
}

cudaError_t launch_fp8_pack_weight(const void* W, bool f32, int E, int N, int K, uint8_t* codes, float* scales,
                                   cudaStream_t s) {
  const int NB = (N + kFp8Block - 1) / kFp8Block, KB = (K + kFp8Block - 1) / kFp8Block;
  const long long grid = static_cast<long long>(E) * NB * KB;
  if (grid > 0x7FFFFFFFLL) return cudaErrorInvalidConfiguration;
  if (f32)
    fp8_pack_weight_kernel<true><<<static_cast<unsigned>(grid), kThreads, 0, s>>>(W, N, K, NB, KB, codes, scales);
  else
    fp8_pack_weight_kernel<false><<<static_cast<unsigned>(grid), kThreads, 0, s>>>(W, N, K, NB, KB, codes, scales);
  return cudaGetLastError();
}

}  // namespace biloco
