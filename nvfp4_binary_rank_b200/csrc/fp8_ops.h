// Host-side declarations of the FP8 block-format operators and the block norm.
#pragma once

#include <cstddef>
#include <cstdint>
#include <utility>

#include <cuda_runtime.h>

namespace biloco {

// Launch with programmatic stream serialisation: the grid may start while the kernel
// before it on the stream finishes.  Every kernel launched this way waits for that
// kernel (griddepcontrol.wait) before it reads anything but weights.
template <typename... P, typename... A>
cudaError_t launch_pdl(void (*kernel)(P...), unsigned grid, unsigned threads, size_t smem, unsigned cluster,
                       cudaStream_t s, A&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.numAttrs = 1;
  if (cluster > 1) {
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.numAttrs = 2;
  }
  cfg.attrs = attr;
  return cudaLaunchKernelEx(&cfg, kernel, P(args)...);
}

cudaError_t launch_fp8_quant_act(const uint16_t* x, long long ldx, int M, int K, uint8_t* codes, float* scales,
                                 cudaStream_t s);
cudaError_t launch_fp8_pack_weight(const void* W, bool f32, int E, int N, int K, uint8_t* codes, float* scales,
                                   cudaStream_t s);

// Validated arguments; returns a BILOCO_* status.
int run_fp8_gemm(const uint8_t* xq, const float* xs, const uint8_t* wq, const float* ws, void* y, bool y_f32, int M,
                 int N, int K, cudaStream_t s);

struct BlockNormArgs {
  const uint16_t* y;        // [M][D] bf16, row stride ldy; may be null
  const void* h;            // [M][D] bf16 or FP32, row stride ldh; may be null
  const void* post_w;       // [D] or null
  const void* gate;         // [G][D] or null
  const void* pre_w;        // [D] or null
  void* h_out;              // [M][D] of h's type, row stride ldho; may be null
  uint16_t* x_out;          // [M][D] bf16, or null
  uint8_t* codes;           // [M][D] E4M3, or null
  float* scales;            // [ceil(D/128)][M]
  long long ldy, ldh, ldho;
  float res_scale, offset, eps;
  int M, D, rows_per_gate;
  bool h_f32, w_f32, gate_f32;
};
cudaError_t launch_block_norm(const BlockNormArgs& a, cudaStream_t s);

}  // namespace biloco
