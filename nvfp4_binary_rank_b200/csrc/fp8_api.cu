// C ABI of the FP8 block-format operators and the block norm: argument checks only.
#include <cstdint>

#include <cuda_runtime.h>

#include "../../include/biloco.h"
#include "fp8_dev.cuh"
#include "fp8_moe.h"
#include "fp8_ops.h"
#include "internal.h"

using namespace biloco;

namespace {

bool off(const void* p, unsigned bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) != 0; }

int status_of(cudaError_t e) { return e == cudaSuccess ? BILOCO_OK : BILOCO_ERR_CUDA; }

bool bad_type(int t) { return t != BILOCO_TYPE_BF16 && t != BILOCO_TYPE_F32; }

constexpr int kMaxDim = 1 << 24, kMaxRows = 1 << 30;

}  // namespace

extern "C" {

int biloco_fp8_quant_act(const void* x_bf16, long long ldx, int M, int K, uint8_t* codes, float* scales,
                         biloco_stream_t stream) {
  if (M < 0 || (M > 0 && (!x_bf16 || !codes || !scales))) return BILOCO_ERR_ARG;
  if (K < 16 || K % 16 || K > kMaxDim || ldx < K || ldx % 8 || M > kMaxRows) return BILOCO_ERR_SHAPE;
  if (static_cast<long long>(M) * ((K + 511) / 512) > 0x7FFFFFFFLL) return BILOCO_ERR_SHAPE;
  if (off(x_bf16, 16) || off(codes, 16) || off(scales, 4)) return BILOCO_ERR_ALIGN;
  const int d = check_device();
  if (d || M == 0) return d;
  return status_of(launch_fp8_quant_act(static_cast<const uint16_t*>(x_bf16), ldx, M, K, codes, scales,
                                        reinterpret_cast<cudaStream_t>(stream)));
}

int biloco_fp8_pack_weight(const void* W, int w_type, int E, int N, int K, uint8_t* codes, float* scales,
                           biloco_stream_t stream) {
  if (!W || !codes || !scales || bad_type(w_type)) return BILOCO_ERR_ARG;
  if (E < 1 || N < 1 || K < 16 || K % 16 || K > kMaxDim || N > kMaxDim) return BILOCO_ERR_SHAPE;
  if (static_cast<long long>(E) * ((N + 127) / 128) * ((K + 127) / 128) > 0x7FFFFFFFLL) return BILOCO_ERR_SHAPE;
  if (off(W, 16) || off(codes, 16) || off(scales, 4)) return BILOCO_ERR_ALIGN;
  const int d = check_device();
  if (d) return d;
  return status_of(launch_fp8_pack_weight(W, w_type == BILOCO_TYPE_F32, E, N, K, codes, scales,
                                          reinterpret_cast<cudaStream_t>(stream)));
}

int biloco_fp8_gemm(const uint8_t* x_codes, const float* x_scales, const uint8_t* w_codes, const float* w_scales,
                    void* y, int y_type, int M, int N, int K, biloco_stream_t stream) {
  if (M < 0 || bad_type(y_type) || !w_codes || !w_scales || (M > 0 && (!x_codes || !x_scales || !y)))
    return BILOCO_ERR_ARG;
  if (N < 1 || K < 16 || K % 16 || K > kMaxDim || N > kMaxDim || M > kMaxDim) return BILOCO_ERR_SHAPE;
  if (off(x_codes, 16) || off(w_codes, 16) || off(x_scales, 4) || off(w_scales, 4) ||
      off(y, y_type == BILOCO_TYPE_F32 ? 4 : 2))
    return BILOCO_ERR_ALIGN;
  const int d = check_device();
  if (d || M == 0) return d;
  return run_fp8_gemm(x_codes, x_scales, w_codes, w_scales, y, y_type == BILOCO_TYPE_F32, M, N, K,
                      reinterpret_cast<cudaStream_t>(stream));
}

int biloco_selftest_drop_scales(void) {
  fp8_drop_scales();
  return BILOCO_OK;
}

int biloco_block_norm(const void* y_bf16, long long ldy, const void* h, long long ldh, int h_type,
                      const void* post_weight, const void* pre_weight, int w_type, const void* gate, int gate_type,
                      int gate_rows, float res_scale, float offset, float eps, int M, int D, void* h_out,
                      long long ldho, void* x_bf16, uint8_t* codes, float* scales, biloco_stream_t stream) {
  if (M < 0 || bad_type(h_type) || bad_type(w_type) || bad_type(gate_type)) return BILOCO_ERR_ARG;
  if ((!y_bf16 && !h) || (!y_bf16 && (post_weight || gate)) || (!h_out && !x_bf16 && !codes) ||
      ((x_bf16 || codes) && !pre_weight) || (pre_weight && !x_bf16 && !codes) || (!codes != !scales))
    return M == 0 ? BILOCO_OK : BILOCO_ERR_ARG;
  if (D < 8 || D % 8 || D > BILOCO_NORM_MAX_D || (codes && D % 16) || M > kMaxRows) return BILOCO_ERR_SHAPE;
  if ((y_bf16 && (ldy < D || ldy % 8)) || (h && (ldh < D || ldh % 8)) || (h_out && (ldho < D || ldho % 8)))
    return BILOCO_ERR_SHAPE;
  if (gate && (gate_rows < 1 || M % gate_rows)) return BILOCO_ERR_SHAPE;
  if (off(y_bf16, 16) || off(h, 16) || off(post_weight, 16) || off(pre_weight, 16) || off(gate, 16) ||
      off(h_out, 16) || off(x_bf16, 16) || off(codes, 16) || off(scales, 4))
    return BILOCO_ERR_ALIGN;
  const int d = check_device();
  if (d || M == 0) return d;
  BlockNormArgs a = {};
  a.y = static_cast<const uint16_t*>(y_bf16);
  a.h = h;
  a.post_w = post_weight;
  a.gate = gate;
  a.pre_w = pre_weight;
  a.h_out = h_out;
  a.x_out = static_cast<uint16_t*>(x_bf16);
  a.codes = codes;
  a.scales = scales;
  a.ldy = ldy;
  a.ldh = ldh;
  a.ldho = ldho;
  a.res_scale = res_scale;
  a.offset = offset;
  a.eps = eps;
  a.M = M;
  a.D = D;
  a.rows_per_gate = gate ? M / gate_rows : 1;
  a.h_f32 = h_type == BILOCO_TYPE_F32;
  a.w_f32 = w_type == BILOCO_TYPE_F32;
  a.gate_f32 = gate_type == BILOCO_TYPE_F32;
  return status_of(launch_block_norm(a, reinterpret_cast<cudaStream_t>(stream)));
}

size_t biloco_fp8_moe_workspace_bytes(int T, int D, int F, int k, int shared) {
  if (T < 1 || T > BILOCO_MOE_MAX_T || D < 16 || D % 16 || D > BILOCO_MOE_MAX_D || F < 16 || F % 16 ||
      F > BILOCO_MOE_MAX_F || k < 1 || k > BILOCO_MOE_MAX_K || shared < 0 || shared > BILOCO_MOE_MAX_SHARED)
    return 0;
  MoeArgs a = {};
  a.T = T;
  a.D = D;
  a.F = F;
  a.k = k;
  a.shared = shared;
  return moe_carve(a, nullptr);
}

int biloco_fp8_moe(const void* x_bf16, long long ldx, const void* router, int router_type, const float* bias,
                   const uint8_t* w13_codes, const float* w13_scales, const uint8_t* w2_codes, const float* w2_scales,
                   int T, int D, int F, int E, int k, int shared, int score, int renorm, float route_scale,
                   void* y_bf16, int* ids, float* weights, void* workspace, size_t workspace_bytes,
                   biloco_stream_t stream) {
  if (T < 0 || bad_type(router_type) || (score != BILOCO_SCORE_SOFTMAX && score != BILOCO_SCORE_SIGMOID))
    return BILOCO_ERR_ARG;
  if (T == 0) return BILOCO_OK;
  if (!x_bf16 || !router || !w13_codes || !w13_scales || !w2_codes || !w2_scales || !y_bf16 || !ids || !weights ||
      !workspace)
    return BILOCO_ERR_ARG;
  const size_t need = biloco_fp8_moe_workspace_bytes(T, D, F, k, shared);
  if (!need || E < 1 || E > BILOCO_MOE_MAX_E || k > E || ldx < D || ldx % 8) return BILOCO_ERR_SHAPE;
  if (workspace_bytes < need) return BILOCO_ERR_ARG;
  if (off(x_bf16, 16) || off(router, 16) || off(bias, 4) || off(w13_codes, 16) || off(w13_scales, 4) ||
      off(w2_codes, 16) || off(w2_scales, 4) || off(y_bf16, 8) || off(ids, 4) || off(weights, 4) || off(workspace, 256))
    return BILOCO_ERR_ALIGN;
  const int d = check_device();
  if (d) return d;
  MoeArgs a = {};
  a.x = static_cast<const uint16_t*>(x_bf16);
  a.router = router;
  a.bias = bias;
  a.w13 = w13_codes;
  a.s13 = w13_scales;
  a.w2 = w2_codes;
  a.s2 = w2_scales;
  a.y = static_cast<uint16_t*>(y_bf16);
  a.ids = ids;
  a.weights = weights;
  a.ldx = ldx;
  a.T = T;
  a.D = D;
  a.F = F;
  a.E = E;
  a.k = k;
  a.shared = shared;
  a.sigmoid = score == BILOCO_SCORE_SIGMOID;
  a.renorm = renorm != 0;
  a.router_f32 = router_type == BILOCO_TYPE_F32;
  a.route_scale = route_scale;
  moe_carve(a, static_cast<uint8_t*>(workspace));
  return status_of(launch_fp8_moe(a, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
