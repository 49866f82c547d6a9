/*
 * biloco.h - C ABI of libbiloco.so: the fused NVFP4 GEMM with a binary-sign
 * low-rank correction on one B200 (sm_100a).
 *
 * The operation (BiLoCo README, github jindavid/BiLoCo, sections "Decomposition"
 * and "Kernel"): a weight is split as W ~= U diag(alpha) V^T + R with sign
 * factors U in {+-1}^{N x r}, V in {+-1}^{K x r} and an NVFP4 residual R, and the
 * layer output is
 *
 *     y = FP4(x) FP4(R)^T + sum_i alpha_i (x . v_i) u_i            (BF16 out)
 *
 * computed in one fused launch: the FP4 product on the tensor cores, the sign
 * correction on the CUDA cores.
 *
 * Conventions for every call
 *   - Pointers are DEVICE pointers owned by the caller unless stated otherwise;
 *     the library never frees them.  Calls are asynchronous and ordered on
 *     `stream` (NULL = the legacy default stream).
 *   - Return value: BILOCO_OK (0) or a negative BILOCO_ERR_* code.  Argument,
 *     shape and alignment errors are detected on the host before anything is
 *     launched.  Errors raised inside a kernel (a bounded wait that expired)
 *     are reported by biloco_last_error().
 *   - Row-major everywhere.  "x_bf16" and "y_bf16" point to IEEE bfloat16 data.
 *   - The library keeps scratch memory per (device, stream), allocated on first
 *     use and grown when a larger shape arrives; biloco_shutdown() frees it.
 *     Calls on one stream must not run concurrently with each other from
 *     several host threads.
 *
 * NVFP4 format used throughout (E2M1 elements, one E4M3 scale per 16 elements
 * along K):
 *   - element codes: 4-bit E2M1, grid {0, +-0.5, +-1, +-1.5, +-2, +-3, +-4, +-6};
 *     element 2j of a row in the low nibble of byte j; a zero is always code 0.
 *   - scale s = E4M3(amax_block / 6) for activations (no tensor scale), and
 *     s = E4M3(amax_block / (6 g)) for the weight with g = amax(|R|) / 2688
 *     (g = 1 if R == 0); E4M3 rounding is nearest-even with saturation at 448.
 *   - code = E2M1(v / S), S = s (activation) or S = s * g (weight), FP32
 *     division rounded to nearest, E2M1 nearest with ties to the even code,
 *     |v/S| > 6 saturates; if S == 0 the block's codes are 0.
 *
 * Sign packing: bit 1 = -1, bit 0 = +1 (a zero counts as +1), least significant
 * bit first in little-endian uint32 words; unused tail bits are 0.
 */
#ifndef BILOCO_H
#define BILOCO_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Same object as cudaStream_t. */
typedef struct CUstream_st *biloco_stream_t;

enum {
  BILOCO_OK = 0,
  BILOCO_ERR_ARG = -1,     /* NULL pointer where one is required, negative size  */
  BILOCO_ERR_SHAPE = -2,   /* shape outside the supported limits                  */
  BILOCO_ERR_ALIGN = -3,   /* pointer not 16-byte aligned                         */
  BILOCO_ERR_CUDA = -4,    /* a CUDA runtime call or a kernel launch failed       */
  BILOCO_ERR_TIMEOUT = -5, /* a bounded device-side wait expired (see last_error) */
  BILOCO_ERR_NOMEM = -6,   /* library scratch could not be allocated              */
  BILOCO_ERR_DEVICE = -7,  /* the current device is not an sm_100 GPU             */
  BILOCO_ERR_RESIDENCY = -8 /* the GEMM grid cannot be resident on the GPU at once  */
};

/* Size limits of biloco_gemm.  The weight is cut into (N/128) * ceil(K/256) units
 * of 128 rows x 256 elements; at most BILOCO_MAX_UNITS of them (16.7 M units is
 * 275 GB of codes, more than any single GPU holds). */
#define BILOCO_MAX_M 128
#define BILOCO_MAX_R 1024
#define BILOCO_MAX_N (1 << 24)
#define BILOCO_MAX_UNITS (1 << 24)

/* z schedules of biloco_gemm (BiLoCo README, section "Kernel", mode table):
 *   BILOCO_MODE_AUTO       pick per (M, r, K) from a measured table
 *   BILOCO_MODE_SHARED_Z   every CTA computes one slice of z = alpha . (V^T x) at
 *                          entry and publishes it to scratch behind an arrival
 *                          counter; the GEMM tiles read z in their epilogue
 *                          (the "side CTAs + arrival flag" schedule)
 *   BILOCO_MODE_LOCAL_Z    every CTA computes, at entry, the part of z that its own
 *                          tiles need; no cross-CTA exchange (the "every CTA computes
 *                          the correction at kernel entry" schedule) */
enum { BILOCO_MODE_AUTO = 0, BILOCO_MODE_SHARED_Z = 1, BILOCO_MODE_LOCAL_Z = 2 };

/*
 * biloco_quant_act - BF16 activation -> NVFP4 codes and E4M3 block scales.
 * (BiLoCo README, section "Kernel": the activation enters the FP4 product as
 * NVFP4 codes A plus block scales A_sf; no tensor scale is passed.)
 *
 *   x_bf16  [M][K] bfloat16, 16-byte aligned
 *   M, K    M >= 1, K >= 16, K % 16 == 0
 *   x_fp4   out [M][K/2] bytes (two codes per byte)
 *   x_sf    out [M][K/16] E4M3 bytes
 * Bit-exact with the rules in the header comment.
 */
int biloco_quant_act(const void *x_bf16, int M, int K, uint8_t *x_fp4, uint8_t *x_sf,
                     biloco_stream_t stream);

/*
 * biloco_pack_signs - +-1 matrix -> packed sign words.
 * (BiLoCo README, section "Kernel": pack_signs(V.T), pack_signs(U.T).)
 *
 *   S     [rows][cols] float; bit = 1 where S < 0
 *   bits  out [rows][ceil(cols/32)] uint32, bit j of word w <-> column 32w + j
 * For the GEMM: Vbits = pack_signs(V^T) with rows = r, cols = K, and
 * Ubits = pack_signs(U) with rows = N, cols = r.
 */
int biloco_pack_signs(const float *S, int rows, int cols, uint32_t *bits,
                      biloco_stream_t stream);

/*
 * biloco_pack_weight - FP32 residual R -> NVFP4 codes, block scales in the
 * GEMM's tile layout, and the FP32 tensor scale.
 * (BiLoCo README, section "Decomposition": R is quantised to NVFP4; section
 * "Kernel": W_fp4, W_sf, w_global_scale.)
 *
 *   R       [N][K] float, 16-byte aligned; N % 128 == 0, K % 64 == 0
 *   W_fp4   out [N][K/2] bytes, 16-byte aligned
 *   W_sf    out biloco_weight_sf_bytes(N, K) bytes, 16-byte aligned, tile layout:
 *           the scale of weight row n and 16-element block b (k = 16b .. 16b+15)
 *           sits at byte
 *              ((((n/128) * KC + b/16) * 4 + (b%16)/4) * 512)
 *              + (n%32) * 16 + ((n%128)/32) * 4 + (b%4)
 *           with KC = ceil(K/256); bytes past K are zero.
 *   gscale  out device float, the tensor scale g
 * Runs three kernels; needs no host synchronisation.
 */
int biloco_pack_weight(const float *R, int N, int K, uint8_t *W_fp4, uint8_t *W_sf,
                       float *gscale, biloco_stream_t stream);

/* Bytes of the weight scale array: N * ceil(K/256) * 16. */
size_t biloco_weight_sf_bytes(int N, int K);

/*
 * biloco_decompose - W ~= U diag(alpha) V^T + R with binary sign factors.
 * (BiLoCo README, section "Decomposition": each rank-one term starts from random
 * signs and alternates u = sign(R v), v = sign(R^T u) for T steps, takes the
 * Frobenius-optimal coefficient and deflates the residual; after all r terms the
 * coefficients are refit jointly by least squares for the fixed signs.)
 *
 *   W          [N][K] float, 4-byte aligned, not modified (R_out may alias it)
 *   r, T       0 <= r <= 1024 terms, T >= 1 alternations per term
 *   v0bits     [r][ceil(K/32)] uint32: the start signs of each term's v, packed
 *              like pack_signs (bit 1 = -1); the caller draws them (the README
 *              seeds a generator); may be NULL when r == 0
 *   Ubits      out [N][ceil(r/32)] uint32 = pack_signs(U)    (biloco_gemm's Ubits)
 *   Vbits      out [r][ceil(K/32)] uint32 = pack_signs(V^T)  (biloco_gemm's Vbits)
 *   alpha      out [r] float, the refit coefficients
 *   R_out      out [N][K] float, W - U diag(alpha) V^T (feed it to
 *              biloco_pack_weight for the NVFP4 residual)
 *   workspace  device memory of at least biloco_decompose_workspace_bytes(N, K, r)
 *              bytes, 256-byte aligned, owned by the caller (it holds the FP64
 *              residual: about 8 N K bytes)
 * Every sign is decided on an FP64 sum, with sign(0) = +1; alpha_i = u^T R v /
 * (N K) for the current residual; the refit solves the normal equations
 * (u_i . u_j)(v_i . v_j) alpha = u_i^T W v_i by conjugate gradients (the
 * minimum-norm solution if terms repeat).  Asynchronous on `stream`; about
 * r (3 T + 2) kernel launches.  Errors: BILOCO_ERR_ARG (NULL pointer, workspace
 * too small), _SHAPE (N, K < 1, r out of range, T < 1, N K > 2^31), _ALIGN,
 * _DEVICE, _CUDA.
 */
size_t biloco_decompose_workspace_bytes(int N, int K, int r);
int biloco_decompose(const float *W, int N, int K, int r, int T, const uint32_t *v0bits,
                     uint32_t *Ubits, uint32_t *Vbits, float *alpha, float *R_out,
                     void *workspace, size_t workspace_bytes, biloco_stream_t stream);

/*
 * biloco_gemm - y = FP4(x) FP4(R)^T + sum_i alpha_i (x . v_i) u_i, in BF16.
 * (BiLoCo README, section "Kernel": one launch for decode batches; the FP4 GEMM
 * on tensor cores, z = alpha . (V x) on CUDA cores from bit-packed V, U z expanded
 * in the GEMM epilogue before the BF16 store.)
 *
 *   x_bf16  [M][K] bfloat16 activation; quantised inside the call exactly like
 *           biloco_quant_act, and used unquantised (BF16) for the correction
 *   W_fp4, W_sf, gscale   as written by biloco_pack_weight
 *   Ubits   [N][ceil(r/32)] uint32 = pack_signs(U)      (may be NULL when r == 0)
 *   Vbits   [r][K/32] uint32 = pack_signs(V^T)           (may be NULL when r == 0)
 *   alpha   [r] float                                    (may be NULL when r == 0)
 *   y_bf16  out [M][N] bfloat16, rounded to nearest-even from FP32
 *   limits  1 <= M <= 128, N % 128 == 0, N <= 2^24, K % 64 == 0, 0 <= r <= 1024,
 *           (N/128) * ceil(K/256) <= 2^24
 * Accumulation is FP32 in an unspecified order; results are deterministic for a
 * fixed shape, mode and GPU.  Under the shared-z schedule, batches of up to 128
 * rows run one kernel that quantises the activation itself when each CTA's share
 * of the weight fits the batch class (ceil(units / G) <= 16 units of 128 x 256
 * up to 16 rows, <= 64 above); otherwise an activation quantiser runs first for
 * M > 8 (biloco_gemm_kernel_count).
 * The fused kernel is launched with programmatic dependent launch: it may start
 * while the kernel before it on the stream finishes, and it reads W_fp4 and
 * W_sf before waiting for that kernel (everything else after).  So the weight
 * operand must not be written by a preceding kernel that triggers early launch
 * of its dependents (griddepcontrol.launch_dependents); kernels without that
 * trigger, biloco_pack_weight's included, are fully ordered before the call.
 *
 * Residency: the GEMM kernel runs one CTA per SM on G <= min(#SMs, units) CTAs
 * that exchange data behind grid-wide arrival counters, so all G CTAs must be
 * resident together.  The host checks that one CTA per SM fits
 * (BILOCO_ERR_RESIDENCY otherwise).  With the default launch form
 * (BILOCO_LAUNCH_PDL) the GPU must also not be shared with long-running kernels
 * on other streams, or with another biloco_gemm call running concurrently on
 * another stream: CTAs that cannot start leave the others waiting, and after
 * their bounded wait (about 1 s) they give up and biloco_last_error reports
 * BILOCO_ERR_TIMEOUT (y is then not valid).  Where the GPU is shared, select
 * BILOCO_LAUNCH_COOPERATIVE (biloco_set_launch): the driver then starts the
 * grid only once all of its CTAs can be resident.
 */
int biloco_gemm(const void *x_bf16, const uint8_t *W_fp4, const uint8_t *W_sf,
                const float *gscale, const uint32_t *Ubits, const uint32_t *Vbits,
                const float *alpha, void *y_bf16, int M, int N, int K, int r,
                biloco_stream_t stream);

/*
 * biloco_gemm_noalloc - biloco_gemm with no device allocation.
 * The BiLoCo pages have no counterpart of this call: it exists for callers that
 * cannot let the library allocate, e.g. an engine that has reserved nearly all of
 * HBM for its own pools, or a decode loop that cannot have its stream stalled
 * while biloco_gemm grows its per-stream scratch (synchronise, free, cudaMalloc).
 *
 * Same arguments, limits, results and error codes as biloco_gemm; the results
 * equal biloco_gemm's for the same shape and mode.  Its scratch is one static
 * device array of BILOCO_NOALLOC_SCRATCH_BYTES per device, part of the library's
 * device code; the call never calls cudaMalloc or cudaFree.  Extra limits,
 * checked on the host before anything is launched (BILOCO_ERR_SHAPE otherwise):
 *   N <= BILOCO_NOALLOC_MAX_N, and the call's scratch fits the array.  That
 *   scratch is 16 896 bytes of status and counters plus, each rounded up to 256,
 *   with KC = ceil(K/256), G = min(#SMs, (N/128)*KC) (for 65..128 rows on the
 *   decode-batch kernel at most 5*(N/128)/2 where that keeps <= 64 units per
 *   CTA) and rpad = 16*ceil(r/16):
 *   decode-batch kernel (M <= 128, shared-z schedule, ceil(units/G) <= 16 for
 *   M <= 16 or <= 64 above; BN = 16 for M <= 16, else the batch class 32, 64
 *   or 128 that holds M):
 *     KC * (M <= 16 ? 2304 : BN * 128 + 2048)  (quantised activation image)
 *     ztile + max(G, ceil(r/128)) * BN * 512   (z tiles, V-side partial sums;
 *                                               ztile = 65536 for M <= 16,
 *                                               else 4096 * BN)
 *     M * rpad * 4                             (z)
 *     2 * G * BN * 512                         (split-K partials)
 *   general kernel (every other shape; BN = 16, 32, 64, 128 for M <= 16, 32,
 *   64, 128):
 *     M > 8:  M*K/2 + KC*2048                  (quantised activation)
 *     r > 0:  (KC + 1) * M * rpad * 4          (z partials and z)
 *     always: 2 * G * BN * 512                 (split-K partials)
 *   On a 148-SM B200 every M <= 64 shape with K <= 13824 and r <= 1024 fits;
 *   M > 64 fits only small weights (few units, so a small G).
 * Caveats:
 *   - There is one array per device, shared by all streams and host threads:
 *     calls that overlap in time (on different streams, or from several threads
 *     without ordering) race on it and give wrong results.  Order the calls.
 *   - The first call on a device looks up the array's address
 *     (cudaGetSymbolAddress) and clears its status and counters with an
 *     asynchronous memset; make it before any stream capture begins.
 *   - Device-side errors (an expired bounded wait) are reported by
 *     biloco_last_error(stream), which also clears the array's counters.
 */
#define BILOCO_NOALLOC_SCRATCH_BYTES (16u << 20)
#define BILOCO_NOALLOC_MAX_N (1 << 18)
int biloco_gemm_noalloc(const void *x_bf16, const uint8_t *W_fp4, const uint8_t *W_sf,
                        const float *gscale, const uint32_t *Ubits, const uint32_t *Vbits,
                        const float *alpha, void *y_bf16, int M, int N, int K, int r,
                        biloco_stream_t stream);

/*
 * ---- FP8 block format -----------------------------------------------------
 * The layers of a model that stay at 8 bits next to the NVFP4 ones, and the steps
 * between them, for inference: none has a backward pass.  The BiLoCo pages have no
 * counterpart of these calls.
 *
 * Format: E4M3 codes (sign, 4 exponent, 3 mantissa bits; 0x7F and 0xFF are NaN) with
 * one FP32 scale per 128 elements of a row (activations) or per 128 x 128 tile
 * (weights); the last block of a row, or tile, may be smaller.
 *     a = max(max |v| over the block, 2^-100)
 *     scale = RN(a / 448),  code = E4M3(RN(v * RN(448 / a)))
 * in FP32, E4M3 to nearest-even with saturation at 448.  A NaN makes its whole block
 * NaN; an infinity makes the block's scale infinite (and its values NaN).
 *
 * Types of a floating array where a call takes more than one:
 */
enum { BILOCO_TYPE_BF16 = 0, BILOCO_TYPE_F32 = 1 };

/*
 * biloco_fp8_quant_act - BF16 activation -> FP8 blocks.
 *   x_bf16  [M][K] bfloat16, row stride ldx elements, 16-byte aligned; ldx % 8 == 0
 *   M, K    0 <= M <= 2^30 (0: nothing is done), K >= 16, K % 16 == 0, M ceil(K/512) < 2^31
 *   codes   out [M][K] E4M3 bytes, 16-byte aligned
 *   scales  out [ceil(K/128)][M] float (block-major: one token's scales are M apart)
 */
int biloco_fp8_quant_act(const void *x_bf16, long long ldx, int M, int K, uint8_t *codes,
                         float *scales, biloco_stream_t stream);

/*
 * biloco_fp8_pack_weight - E weights of [N][K] (contiguous, BF16 or FP32) -> FP8 tiles.
 *   codes   out [E][N][K] E4M3 bytes
 *   scales  out [E][ceil(N/128)][ceil(K/128)] float
 * K % 16 == 0; W and codes 16-byte aligned.  Tiles do not cross weights.
 */
int biloco_fp8_pack_weight(const void *W, int w_type, int E, int N, int K, uint8_t *codes,
                           float *scales, biloco_stream_t stream);

/*
 * biloco_fp8_gemm - y[m,n] = sum_b xs[b,m] ws[n/128,b] sum_{k in block b} x[m,k] w[n,k].
 *   x_codes [M][K], x_scales [ceil(K/128)][M]   as written by biloco_fp8_quant_act
 *   w_codes [N][K], w_scales [ceil(N/128)][ceil(K/128)]  as by biloco_fp8_pack_weight
 *   y       out [M][N], BF16 (2-byte aligned) or FP32 (4-byte aligned) by y_type
 *   limits  0 <= M <= 2^24 (0: nothing is done), 1 <= N <= 2^24, K % 16 == 0,
 *           16 <= K <= 2^24; codes 16-byte aligned
 * Any batch size runs one kernel, which keeps no scratch and shares nothing between
 * calls: calls on different streams, and graphs replayed at once, do not disturb each
 * other.  Sums are FP32; the result depends only on the operands, the shape and the GPU
 * (K is split by how many clusters of CTAs it holds at once).  The product of two scales
 * is formed first, in FP32: beyond 2^128 it is infinite, below 2^-126 it loses bits.
 * The kernel is launched with programmatic dependent launch and reads w_codes before it
 * waits for the kernel before it (see biloco_gemm on what must not write the weight: of
 * this library's calls only the packers may have written it since the last kernel of
 * another origin on the stream).
 * A bounded wait that expires inside the kernel is reported by biloco_last_error on the
 * call's stream; y is then not valid.  That of a call captured into a graph, or on a
 * stream beyond the first 1023 that made such calls on the device, is reported on whichever
 * stream asks first.
 */
int biloco_fp8_gemm(const uint8_t *x_codes, const float *x_scales, const uint8_t *w_codes,
                    const float *w_scales, void *y, int y_type, int M, int N, int K,
                    biloco_stream_t stream);

/*
 * biloco_block_norm - the step between two blocks of a layer, in one pass:
 *     u  = y rsqrt(mean(y^2) + eps) (post_weight + offset)     (u = y without post_weight)
 *     h' = res_scale h + gate u
 *     x  = h' rsqrt(mean(h'^2) + eps) (pre_weight + offset)
 *   y_bf16       [M][D] bfloat16 output of the block, row stride ldy; NULL: no block
 *                before (u = 0, no post_weight, no gate)
 *   h            [M][D] residual stream of type h_type, row stride ldh; NULL: none yet
 *   post_weight, pre_weight   [D] of type w_type, NULL: no norm after / before
 *   gate         [gate_rows][D] of gate_type, row m takes row m / (M / gate_rows)
 *                (M % gate_rows == 0); NULL: 1
 *   h_out        out [M][D] of type h_type, row stride ldho; may be h itself, or NULL
 *   x_bf16       out [M][D] bfloat16, or NULL
 *   codes,scales out x as FP8 blocks (D % 16 == 0), layout of biloco_fp8_quant_act, or NULL
 * h' enters x unrounded, and x the FP8 blocks unrounded: each output is rounded once.
 * A row's FP32 sums may be added in another order in a batch of another size.
 * limits: 0 <= M <= 2^30, 8 <= D <= BILOCO_NORM_MAX_D, D % 8 == 0, row strides >= D and multiples of 8
 * elements, 16-byte aligned arrays.  Outputs must not overlap inputs other than h_out = h
 * with the same stride.
 */
#define BILOCO_NORM_MAX_D 32768
int biloco_block_norm(const void *y_bf16, long long ldy, const void *h, long long ldh, int h_type,
                      const void *post_weight, const void *pre_weight, int w_type,
                      const void *gate, int gate_type, int gate_rows, float res_scale,
                      float offset, float eps, int M, int D, void *h_out, long long ldho,
                      void *x_bf16, uint8_t *codes, float *scales, biloco_stream_t stream);

/*
 * biloco_fp8_moe - a whole mixture-of-experts layer for a few tokens (up to 64).
 *     score of expert e for token t: softmax over the experts, or sigmoid, of x[t] . router[e]
 *     its k experts: the largest scores (with bias: of score + bias), ties to the lowest index
 *     weight: the score itself (renorm: divided by the sum over the k), times route_scale
 *     y[t] = sum over its experts of weight * W2_e (silu(W1_e x[t]) * (W3_e x[t]))
 *   x_bf16   [T][D] bfloat16, row stride ldx (multiple of 8), not quantised
 *   router   [E][D] of router_type; bias [E] float, for the choice only, or NULL
 *   w13      [E + shared][2F][D] codes and their scales (biloco_fp8_pack_weight on E + shared
 *            weights [2F][D]): rows 0..F-1 are W1 (gate), F..2F-1 are W3 (up)
 *   w2       [E + shared][D][F] codes and scales
 *   shared   the last `shared` experts serve every token with weight 1
 *   y_bf16   out [T][D], 8-byte aligned; ids out [T][k] int, weights out [T][k] float, in the order picked
 *   workspace  device memory of at least biloco_fp8_moe_workspace_bytes (256-byte aligned),
 *            owned by the caller; its contents do not matter before the call and are of no
 *            use after it.  Two calls that may overlap need two of them.
 *   limits   0 <= T <= 64 (0: nothing is done), D and F multiples of 16 up to 16384,
 *            1 <= k <= 16, k <= E <= 512, 0 <= shared <= 4
 * Scores are FP32 sums of eight products each, added with compensation and then in FP64, and
 * compared in FP64; a score that is not a number is picked last.  The products are FP16 x E4M3
 * with FP32 sums (weight scales up to 2^88 keep them finite): rows of x are scaled into FP16
 * exactly (BF16 values more than 2^29 below the row's largest lose bits).  The hidden values
 * are rounded to FP16's 11 bits, where FP32 would hold 24: with a BF16 output the error against
 * an exact layer grows by about 1% (0.00165 to 0.00167 of the output's size).  Those below 2^-28
 * of a token's and expert's largest lose more bits, and below 2^-38 they vanish.  A token with
 * an infinity or NaN spoils only its own row.
 * Four kernels (three for one token) with programmatic dependent launch; router and w2 may be
 * read before the kernel before them on the stream has ended (see biloco_gemm on what must
 * not write the weight: the same as for biloco_fp8_gemm's).
 * The result depends only on the operands, the shape and the GPU (the number of its SMs).
 */
#define BILOCO_MOE_MAX_T 64
#define BILOCO_MOE_MAX_D 16384
#define BILOCO_MOE_MAX_F 16384
#define BILOCO_MOE_MAX_E 512
#define BILOCO_MOE_MAX_K 16
#define BILOCO_MOE_MAX_SHARED 4
enum { BILOCO_SCORE_SOFTMAX = 0, BILOCO_SCORE_SIGMOID = 1 };
size_t biloco_fp8_moe_workspace_bytes(int T, int D, int F, int k, int shared);
int biloco_fp8_moe(const void *x_bf16, long long ldx, const void *router, int router_type,
                   const float *bias, const uint8_t *w13_codes, const float *w13_scales,
                   const uint8_t *w2_codes, const float *w2_scales, int T, int D, int F, int E,
                   int k, int shared, int score, int renorm, float route_scale, void *y_bf16,
                   int *ids, float *weights, void *workspace, size_t workspace_bytes,
                   biloco_stream_t stream);

/*
 * Launch form of the GEMM kernels for later biloco_gemm / biloco_gemm_noalloc
 * calls (process-wide), a combination of:
 *   BILOCO_LAUNCH_PDL          programmatic dependent launch: the kernel may start
 *                              while the kernel before it on the stream finishes
 *                              (its weight stream overlaps that kernel's tail)
 *   BILOCO_LAUNCH_COOPERATIVE  cooperative launch: every CTA of the grid is
 *                              resident together, whatever else runs on the GPU
 * Default BILOCO_LAUNCH_PDL.  With both flags the grid is launched with both
 * attributes where the driver accepts the pair, else cooperative only.  Not part
 * of the BiLoCo pages.  BILOCO_ERR_ARG for unknown flags.
 */
enum { BILOCO_LAUNCH_PDL = 1, BILOCO_LAUNCH_COOPERATIVE = 2 };
int biloco_set_launch(int flags);
int biloco_get_launch(void);

/*
 * Arithmetic of the correction's U side on the CUDA cores (the decode-batch
 * kernel at 1-2 rows; every other shape ignores it), for later calls
 * (process-wide):
 *   BILOCO_CORR_SIGNS  sign-adds: every rank's z added or subtracted per weight row
 *   BILOCO_CORR_LUT    table lookups: each CTA that completes a tile builds, from
 *                      z, the 16 signed sums of every group of four ranks
 *                      (FluxBin, "LUT-based Multiplication"; the BiLoCo README's
 *                      LUT branch), and a weight row adds one entry per four ranks
 *   BILOCO_CORR_AUTO   the measured choice per shape
 * Both give y within the stated tolerance of the oracle (different FP32 summation
 * orders).  BILOCO_ERR_ARG for an unknown value.  Not part of the BiLoCo pages'
 * API.
 */
enum { BILOCO_CORR_AUTO = 0, BILOCO_CORR_SIGNS = 1, BILOCO_CORR_LUT = 2 };
int biloco_set_correction(int arith);
/* The arithmetic biloco_gemm would use for this shape under the current setting. */
int biloco_resolve_correction(int M, int N, int K, int r);

/* Select the z schedule for later biloco_gemm calls (process-wide). */
int biloco_set_mode(int mode);
/* The schedule biloco_gemm would use for this shape under the current setting. */
int biloco_resolve_mode(int M, int N, int K, int r);

/*
 * biloco_last_error - synchronise `stream`, return and clear the first error a
 * kernel on it recorded (BILOCO_ERR_TIMEOUT when a bounded wait expired), or
 * BILOCO_OK.  After an error the stream's scratch counters are reset.  Once
 * biloco_gemm_noalloc has run on the current device, its static scratch is
 * checked and reset the same way; because that array serves every stream, the
 * call then synchronises the whole device first (cudaDeviceSynchronize), so that
 * a no-allocation call still running on another stream is neither missed nor
 * cleared while it runs.  The same holds once a biloco_fp8_gemm call has been captured into
 * a graph.  Where several calls recorded errors, the FP8 product's are kept for the next ask.
 */
int biloco_last_error(biloco_stream_t stream);

/*
 * biloco_selftest_wait_timeout - exercise the failure path on the GPU without a
 * fault.  Launches one warp that waits, through the same bounded mbarrier wait
 * the GEMM kernels use, on a phase nothing completes.  After the wait's
 * wall-clock limit (about 1 s) the kernel records BILOCO_ERR_TIMEOUT in
 * `stream`'s status word and returns, leaving the context usable; a following
 * biloco_last_error(stream) reports it.  The BiLoCo pages have no counterpart
 * of this call.
 */
int biloco_selftest_wait_timeout(biloco_stream_t stream);

/*
 * biloco_selftest_drop_arrivals - exercise the GEMM's own failure path on the GPU
 * without a fault.  The next biloco_gemm or biloco_gemm_noalloc call that runs
 * the decode-batch kernel (M <= 128, shared-z schedule) leaves out the grid-wide
 * arrivals selected by `mask` (1: the z slices, 2: the activation image, which
 * batches of 8 rows and more share, 3: both); every other call, and every call
 * after that one, is unaffected.  The
 * CTAs waiting on those arrivals give up after their bounded wait (about 1 s),
 * leave together, drain their copies and tensor-core work, free their tensor
 * memory and record BILOCO_ERR_TIMEOUT; y of that call is not valid.  A following
 * biloco_last_error(stream) reports the timeout and resets the counters, after
 * which calls on the stream are correct again.  BILOCO_ERR_ARG for a mask outside
 * 0..3.  The BiLoCo pages have no counterpart of this call.
 */
int biloco_selftest_drop_arrivals(int mask);

/*
 * biloco_selftest_drop_scales - the same for biloco_fp8_gemm: in its next call that has
 * rows the block scales never arrive.  The kernel gives up after its bounded wait (about
 * 1 s, and at most another until its last product has ended) and records
 * BILOCO_ERR_TIMEOUT; y of that call is not valid.
 */
int biloco_selftest_drop_scales(void);

/* Human-readable name of a status code (static storage). */
const char *biloco_status_string(int status);

/* Number of kernels biloco_gemm would launch per call for this shape under the
 * current schedule setting: 1 when the GEMM kernel quantises the activation
 * itself (the decode-batch kernel, M <= 128, or the general kernel at M <= 8),
 * else 2 (quantiser + GEMM).  BILOCO_ERR_SHAPE for shapes biloco_gemm rejects.
 * Uses the device's SM count (the current device must be set). */
int biloco_gemm_kernel_count(int M, int N, int K, int r);

/* Free every stream's scratch.  Safe to call more than once. */
void biloco_shutdown(void);

#ifdef __cplusplus
}
#endif
#endif /* BILOCO_H */
