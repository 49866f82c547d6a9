// FP8 product with a scale per block of 128 along K:
//
//   y[m,n] = sum_b sx[b,m] * sw[n/128,b] * sum_{k in block b} xq[m,k] wq[n,k]
//
// Each block's inner sum runs on the tensor cores (tcgen05.mma kind::f8f6f4, four K = 32
// steps) into one of two TMEM accumulators; the promoting warps read it back, multiply
// it by the two scales and add it to FP32 sums in registers while the next block is
// being multiplied into the other accumulator.  Block sums and the running sums are
// FP32; y is rounded once.
//
// Two forms of one kernel:
//   rows form (more than 128 tokens): the MMA's 128 rows are tokens and its columns weight
//     rows, so a thread's scale is one number per block (its token's times its 128
//     columns').  Persistent over tiles; bound by the tensor cores.
//   swapped form (up to 128 tokens): the MMA's 128 rows are weight rows and its columns
//     tokens, so a decode batch is not padded to 128 rows; scales vary over the columns
//     and come through shared memory.  Bound by reading the weight.
// Where there are fewer tiles than CTA slots, a cluster of up to 8 CTAs splits K: each
// leaves its FP32 sums in its own shared memory and the cluster adds them in rank order
// over distributed shared memory, so the result does not depend on timing and no
// workspace or counter outlives the call.
#include <atomic>
#include <cstdint>
#include <mutex>

#include <cuda.h>
#include <cuda_runtime.h>

#include "../../include/biloco.h"
#include "fp8_dev.cuh"
#include "fp8_ops.h"
#include "internal.h"
#include "ptx.cuh"

namespace biloco {

namespace {

__device__ int g_fp8_status;     // first device-side error of an FP8 GEMM on this device

struct Fp8GemmParams {
  const float* xs;       // [KB][M]
  const float* ws;       // [NB][KB]
  void* y;
  int M, N, K, KB, NB;
  int tiles_a, tiles_b;  // tiles along the MMA's rows and columns
  int split;             // CTAs of the cluster that splits K
  int y_f32;
  int vec;               // bytes of the widest aligned store of a y row: 32, 16, 8, 4 or 2
};

// D(tmem) (+)= A(smem) * B(smem)^T, E4M3 operands, FP32 accumulation, M = 128, K = 32.
__device__ __forceinline__ void tc_mma_f8(uint32_t d_tmem, SmemDesc a, SmemDesc b, uint32_t idesc,
                                          uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\t"
      "mov.b64 da, {%1, %2};\n\t"
      "mov.b64 db, {%3, %4};\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], da, db, %5, p;\n\t"
      "}" ::"r"(d_tmem),
      "r"(a.lo), "r"(a.hi), "r"(b.lo), "r"(b.hi), "r"(idesc), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync_all() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
__device__ __forceinline__ uint32_t mapa(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ float ld_dsmem(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr));
  return v;
}

template <bool kSwap, int kBN>
struct Cfg {
  static constexpr int kGroups = kBN > 128 ? 2 : 1;            // promoting warpgroups
  static constexpr int kCols = kBN / kGroups;                  // columns per promoting thread
  static constexpr int kThreads = 128 + 128 * kGroups;
  static constexpr int kCtasPerSm = (kSwap && kBN <= 64) ? 2 : 1;
  static constexpr int kStageBytes = 16384 + kBN * 128;
  static constexpr int kStages = kSwap ? (kBN <= 16 ? 6 : kBN <= 32 ? 5 : kBN <= 64 ? 4 : 6) : (kBN > 128 ? 4 : 6);
  static constexpr int kSmem = kStages * kStageBytes + 1024;   // slack for the 1024-byte alignment
  static constexpr uint32_t kTmemCols = 2 * kBN < 32 ? 32 : 2 * kBN;
  static constexpr int kPitch = kSwap ? 128 : kBN + 4;         // floats per row of the split-K exchange
  static_assert(kStages * kStageBytes >= (kSwap ? kBN : 128) * kPitch * 4, "the exchange reuses the stages");
};

// The tile t of a persistent walk: groups of eight row tiles, column tiles inside, so
// that the tiles in flight share operands in L2.
__device__ __forceinline__ void tile_at(int t, int ta, int tb, int& a, int& b) {
  const int per = 8 * tb, g = t / per, first = g * 8, rows = min(8, ta - first), r = t - g * per;
  a = first + r % rows;
  b = r / rows;
}

// Stores `kCols` consecutive y values of one row.
template <int kCols>
__device__ __forceinline__ void store_row(const Fp8GemmParams& p, long long at, int n_left, const float* v) {
  if (p.y_f32) {
    float* y = static_cast<float*>(p.y) + at;
    if (p.vec >= 16) {
#pragma unroll
      for (int j = 0; j < kCols; j += 4)
        if (j < n_left) *reinterpret_cast<float4*>(y + j) = make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]);
    } else {
#pragma unroll
      for (int j = 0; j < kCols; ++j)
        if (j < n_left) y[j] = v[j];
    }
  } else {
    uint16_t* y = static_cast<uint16_t*>(p.y) + at;
    if (p.vec >= 32) {
#pragma unroll
      for (int j = 0; j < kCols; j += 16)
        if (j < n_left)
          asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(y + j),
                       "r"(bf16x2_from_f32(v[j], v[j + 1])), "r"(bf16x2_from_f32(v[j + 2], v[j + 3])),
                       "r"(bf16x2_from_f32(v[j + 4], v[j + 5])), "r"(bf16x2_from_f32(v[j + 6], v[j + 7])),
                       "r"(bf16x2_from_f32(v[j + 8], v[j + 9])), "r"(bf16x2_from_f32(v[j + 10], v[j + 11])),
                       "r"(bf16x2_from_f32(v[j + 12], v[j + 13])), "r"(bf16x2_from_f32(v[j + 14], v[j + 15]))
                       : "memory");
    } else if (p.vec >= 16) {
#pragma unroll
      for (int j = 0; j < kCols; j += 8)
        if (j < n_left)
          *reinterpret_cast<uint4*>(y + j) =
              make_uint4(bf16x2_from_f32(v[j], v[j + 1]), bf16x2_from_f32(v[j + 2], v[j + 3]),
                         bf16x2_from_f32(v[j + 4], v[j + 5]), bf16x2_from_f32(v[j + 6], v[j + 7]));
    } else {
#pragma unroll
      for (int j = 0; j < kCols; ++j)
        if (j < n_left) y[j] = static_cast<uint16_t>(bf16x2_from_f32(v[j], 0.0f));
    }
  }
}

__device__ __forceinline__ void store_one(const Fp8GemmParams& p, long long at, float v) {
  if (p.y_f32)
    static_cast<float*>(p.y)[at] = v;
  else
    static_cast<uint16_t*>(p.y)[at] = static_cast<uint16_t>(bf16x2_from_f32(v, 0.0f));
}

template <bool kSwap, int kBN>
__global__ void __launch_bounds__(Cfg<kSwap, kBN>::kThreads, Cfg<kSwap, kBN>::kCtasPerSm)
fp8_gemm_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b,
                const Fp8GemmParams p) {
  using C = Cfg<kSwap, kBN>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t bars[2 * C::kStages + 4];
  __shared__ __align__(16) float col_scale[2][kSwap ? kBN : 4];
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_flag;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t smem = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t full0 = smem_u32(bars), empty0 = full0 + 8 * C::kStages;
  const uint32_t tfull0 = empty0 + 8 * C::kStages, tempty0 = tfull0 + 16;

  if (warp == 0 && lane == 0) {
    prefetch_tmap(&tm_a);
    prefetch_tmap(&tm_b);
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(full0 + 8 * i, 1);
      mbar_init(empty0 + 8 * i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(tfull0 + 8 * i, 1);
      mbar_init(tempty0 + 8 * i, 4 * C::kGroups);
    }
    abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&tmem_slot), C::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(&tmem_slot);
  griddep_launch_dependents();

  // this CTA's tiles and its part of K
  const int rank = p.split > 1 ? static_cast<int>(cluster_rank()) : 0;
  const int k0 = static_cast<int>(static_cast<long long>(p.KB) * rank / p.split);
  const int k1 = static_cast<int>(static_cast<long long>(p.KB) * (rank + 1) / p.split);
  const int first = static_cast<int>(blockIdx.x) / p.split, step = static_cast<int>(gridDim.x) / p.split;
  const int tiles = p.tiles_a * p.tiles_b;
  volatile int* const stop = &abort_flag;

  if (warp == 0 && lane == 0) {
    // ---- producer.  The weight tiles of the first stages are requested before the wait
    // for the kernel before this one, which may be writing the activation.
    int pre = 0;
    if (first < tiles) {
      int ta, tb;
      tile_at(first, p.tiles_a, p.tiles_b, ta, tb);
      for (; pre < C::kStages && k0 + pre < k1; ++pre) {
        const uint32_t st = smem + pre * C::kStageBytes;
        mbar_arrive_expect_tx(full0 + 8 * pre, C::kStageBytes);
        if (kSwap) tma_load_2d(st, &tm_a, full0 + 8 * pre, (k0 + pre) * kFp8Block, ta * 128);
        else tma_load_2d(st + 16384, &tm_b, full0 + 8 * pre, (k0 + pre) * kFp8Block, tb * kBN);
      }
    }
    griddep_wait();
    int it = 0;
    bool ok = true;
    for (int t = first; ok && t < tiles; t += step) {
      int ta, tb;
      tile_at(t, p.tiles_a, p.tiles_b, ta, tb);
      for (int kb = k0; kb < k1; ++kb, ++it) {
        const int s = it % C::kStages;
        const uint32_t st = smem + s * C::kStageBytes, bar = full0 + 8 * s;
        const bool done = it < pre;          // its weight tile is on the way
        if (it >= C::kStages && !mbar_wait(empty0 + 8 * s, (it / C::kStages + 1) & 1, stop)) {
          ok = false;
          break;
        }
        if (!done) mbar_arrive_expect_tx(bar, C::kStageBytes);
        if (!(kSwap && done)) tma_load_2d(st, &tm_a, bar, kb * kFp8Block, ta * 128);
        if (kSwap || !done) tma_load_2d(st + 16384, &tm_b, bar, kb * kFp8Block, tb * kBN);
      }
    }
    if (!ok) {
      // give up: wait (bounded) for the copies in flight before the memory is left
      *stop = 1;
      record_error(&g_fp8_status, kDevErrTimeout);
      const int zero = 0;
      for (int j = max(0, it - C::kStages); j < it; ++j)
        mbar_wait(full0 + 8 * (j % C::kStages), (j / C::kStages) & 1, &zero);
    }
  } else if (warp == 1 && lane == 0) {
    // ---- MMA issuer
    const uint32_t idesc = (1u << 4) | (static_cast<uint32_t>(kBN >> 3) << 17) | (8u << 24);
    const SmemDesc a0 = make_sdesc(smem, 16, 1024, 2), b0 = make_sdesc(smem + 16384, 16, 1024, 2);
    int it = 0;
    bool ok = true;
    for (int t = first; ok && t < tiles; t += step) {
      for (int kb = k0; kb < k1; ++kb, ++it) {
        const int s = it % C::kStages, buf = it & 1;
        if ((it >= 2 && !mbar_wait(tempty0 + 8 * buf, (it / 2 + 1) & 1, stop)) ||
            !mbar_wait(full0 + 8 * s, (it / C::kStages) & 1, stop)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t off = static_cast<uint32_t>(s) * (C::kStageBytes >> 4);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          tc_mma_f8(tmem + buf * kBN, sdesc_at(a0, off + 2 * j), sdesc_at(b0, off + 2 * j), idesc, j > 0);
        tc_commit(empty0 + 8 * s);
        tc_commit(tfull0 + 8 * buf);
      }
    }
    if (!ok) {
      *stop = 1;
      record_error(&g_fp8_status, kDevErrTimeout);
      // the products issued last end before the tensor memory is freed (bounded)
      const int zero = 0;
      for (int j = max(0, it - 2); j < it; ++j) mbar_wait(tfull0 + 8 * (j & 1), (j / 2) & 1, &zero);
    }
  } else if (warp >= 4) {
    // ---- promotion: one thread per MMA row and group of kCols columns
    griddep_wait();
    const int grp = (warp - 4) >> 2, row = (warp & 3) * 32 + lane;
    const uint32_t taddr = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + grp * C::kCols;
    int it = 0;
    bool ok = true;
    for (int t = first; ok && t < tiles; t += step) {
      int ta, tb;
      tile_at(t, p.tiles_a, p.tiles_b, ta, tb);
      uint64_t acc[C::kCols / 2];
#pragma unroll
      for (int j = 0; j < C::kCols / 2; ++j) acc[j] = 0;
      // rows form: this row's token and these columns' weight block; swapped form:
      // thread j < kBN holds the scale of column (token) j, and the tile's weight block
      const int wblk = kSwap ? ta : tb * (kBN / 128) + grp;
      const int tok = kSwap ? tb * kBN + row : ta * 128 + row;
      const bool has = tok < p.M && (!kSwap || row < kBN) && wblk < p.NB;
      const float* ps = p.xs + (has ? tok : 0);
      const float* pw = p.ws + static_cast<long long>(has ? wblk : 0) * p.KB;
      auto scale_of = [&](int kb) {
        return has ? __ldg(ps + static_cast<long long>(kb) * p.M) * __ldg(pw + kb) : 0.0f;
      };
      float s_next = k0 < k1 ? scale_of(k0) : 0.0f;
      for (int kb = k0; kb < k1; ++kb, ++it) {
        const float s = s_next;
        if (kb + 1 < k1) s_next = scale_of(kb + 1);
        const int buf = it & 1;
        if (kSwap) {
          if (row < kBN) col_scale[buf][row] = s;
          named_barrier(1, 128);
        }
        if (!mbar_wait(tfull0 + 8 * buf, (it / 2) & 1, stop)) {
          ok = false;
          // the other threads of the group reach their own wait and see the flag
          *stop = 1;
          record_error(&g_fp8_status, kDevErrTimeout);
        }
        if (kSwap ? named_barrier_or(2, 128, !ok) : __any_sync(0xFFFFFFFFu, !ok)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t src = taddr + buf * kBN;
        const uint64_t s2 = f32x2_pack(__float_as_uint(s), __float_as_uint(s));
#pragma unroll
        for (int c = 0; c < C::kCols; c += 16) {
          uint32_t d[16];
          tmem_ld16(src + c, d);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            uint64_t f = s2;
            if (kSwap) f = *reinterpret_cast<const uint64_t*>(&col_scale[buf][(c + 2 * j) % (kSwap ? kBN : 4)]);
            acc[c / 2 + j] = f32x2_fma(f32x2_pack(d[2 * j], d[2 * j + 1]), f, acc[c / 2 + j]);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(tempty0 + 8 * buf);
      }
      float v[C::kCols];
#pragma unroll
      for (int j = 0; j < C::kCols / 2; ++j)
        asm("mov.b64 {%0, %1}, %2;" : "=f"(v[2 * j]), "=f"(v[2 * j + 1]) : "l"(acc[j]));
      if (p.split > 1) {
        // every product of this CTA is done: its stages are free for the exchange
        float* x = reinterpret_cast<float*>(smem_raw + (smem - smem_u32(smem_raw)));
        if (kSwap) {
#pragma unroll
          for (int j = 0; j < C::kCols; ++j) x[j * C::kPitch + row] = v[j];
        } else {
#pragma unroll
          for (int j = 0; j < C::kCols; j += 4)
            *reinterpret_cast<float4*>(x + row * C::kPitch + grp * C::kCols + j) =
                make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]);
        }
      } else if (ok) {
        if (kSwap) {
          const int n = ta * 128 + row;
          if (n < p.N) {
#pragma unroll
            for (int j = 0; j < C::kCols; ++j)
              if (tb * kBN + j < p.M) store_one(p, static_cast<long long>(tb * kBN + j) * p.N + n, v[j]);
          }
        } else {
          const int n = tb * kBN + grp * C::kCols;
          if (tok < p.M && n < p.N) store_row<C::kCols>(p, static_cast<long long>(tok) * p.N + n, p.N - n, v);
        }
      }
    }
  }

  // every role comes here, in the failing case too
  __syncthreads();
  if (p.split > 1) {
    cluster_sync_all();
    // output rows of the exchange: tokens; this CTA finishes rows rank, rank + split, ...
    int ta, tb;
    tile_at(first, p.tiles_a, p.tiles_b, ta, tb);
    const int m0 = kSwap ? tb * kBN : ta * 128, n0 = kSwap ? ta * 128 : tb * kBN;
    constexpr int kRows = kSwap ? kBN : 128, kWide = kSwap ? 128 : kBN;
    const int rows = min(kRows, p.M - m0);
    const bool good = *stop == 0;
    for (int i = tid; i < kWide * ((rows - rank + p.split - 1) / p.split); i += C::kThreads) {
      const int c = i % kWide, r = rank + i / kWide * p.split;
      float sum = 0.0f;
      for (int q = 0; q < p.split; ++q) sum += ld_dsmem(mapa(smem + (r * C::kPitch + c) * 4, q));
      if (good && n0 + c < p.N) store_one(p, static_cast<long long>(m0 + r) * p.N + n0 + c, sum);
    }
    cluster_sync_all();
  }
  __syncwarp();
  if (warp == 1) tmem_dealloc(tmem, C::kTmemCols);
}

template <bool kSwap, int kBN>
cudaError_t launch_instance(const CUtensorMap& ta, const CUtensorMap& tb, Fp8GemmParams& p, cudaStream_t s) {
  using C = Cfg<kSwap, kBN>;
  static std::atomic<unsigned long long> ready{0};       // devices whose shared-memory limit is raised
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = 1ull << (dev & 63);
  if (!(ready.load() & bit)) {
    e = cudaFuncSetAttribute(fp8_gemm_kernel<kSwap, kBN>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return e;
    ready.fetch_or(bit);
  }
  const long long tiles = static_cast<long long>(p.tiles_a) * p.tiles_b;
  const int slots = num_sms() * C::kCtasPerSm;
  int split = 1;
  while (split < 8 && split < p.KB && tiles * (split + 1) <= slots) ++split;
  p.split = split;
  const unsigned grid = static_cast<unsigned>(split > 1 ? tiles * split : tiles < slots ? tiles : slots);
  return launch_pdl(fp8_gemm_kernel<kSwap, kBN>, grid, C::kThreads, C::kSmem, split, s, ta, tb, p);
}

}  // namespace

int fp8_take_status(cudaStream_t s) {
  int status = 0;
  if (cudaMemcpyFromSymbolAsync(&status, g_fp8_status, sizeof(int), 0, cudaMemcpyDeviceToHost, s) != cudaSuccess ||
      cudaStreamSynchronize(s) != cudaSuccess)
    return BILOCO_ERR_CUDA;
  if (status != 0) {
    const int zero = 0;
    if (cudaMemcpyToSymbolAsync(g_fp8_status, &zero, sizeof(int), 0, cudaMemcpyHostToDevice, s) != cudaSuccess ||
        cudaStreamSynchronize(s) != cudaSuccess)
      return BILOCO_ERR_CUDA;
  }
  return status;
}

int run_fp8_gemm(const uint8_t* xq, const float* xs, const uint8_t* wq, const float* ws, void* y, bool y_f32, int M,
                 int N, int K, cudaStream_t s) {
  Fp8GemmParams p = {};
  p.xs = xs;
  p.ws = ws;
  p.y = y;
  p.M = M;
  p.N = N;
  p.K = K;
  p.KB = (K + kFp8Block - 1) / kFp8Block;
  p.NB = (N + 127) / 128;
  p.y_f32 = y_f32;
  const unsigned long long bits = reinterpret_cast<uintptr_t>(y) | static_cast<unsigned long long>(N) * (y_f32 ? 4 : 2);
  p.vec = bits % 32 == 0 ? 32 : bits % 16 == 0 ? 16 : 2;
  const bool swap = M <= 128;
  const int bn = !swap ? 256 : M <= 16 ? 16 : M <= 32 ? 32 : M <= 64 ? 64 : 128;
  p.tiles_a = swap ? p.NB : (M + 127) / 128;
  p.tiles_b = swap ? 1 : (N + bn - 1) / bn;
  if (static_cast<long long>(p.tiles_a) * p.tiles_b > 0x7FFFFFFFLL) return BILOCO_ERR_SHAPE;
  CUtensorMap tx, tw;
  if (!make_tmap(&tx, xq, K, M, swap ? bn : 128) || !make_tmap(&tw, wq, K, N, swap ? 128 : bn)) return BILOCO_ERR_CUDA;
  cudaError_t e;
  if (!swap) e = launch_instance<false, 256>(tx, tw, p, s);
  else if (bn == 16) e = launch_instance<true, 16>(tw, tx, p, s);
  else if (bn == 32) e = launch_instance<true, 32>(tw, tx, p, s);
  else if (bn == 64) e = launch_instance<true, 64>(tw, tx, p, s);
  else e = launch_instance<true, 128>(tw, tx, p, s);
  return e == cudaSuccess ? BILOCO_OK : BILOCO_ERR_CUDA;
}

}  // namespace biloco
