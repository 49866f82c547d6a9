// FP8 product with a scale per block of 128 along K:
//
//   y[m,n] = sum_b sx[b,m] * sw[n/128,b] * sum_{k in block b} xq[m,k] wq[n,k]
//
// Each block's inner sum runs on the tensor cores (tcgen05.mma kind::f8f6f4, four K = 32
// steps) into one of several TMEM accumulators; the promoting warps read it back, multiply
// it by the two scales and add it to FP32 sums in registers while the next blocks are
// being multiplied into the other accumulators.  Block sums and the running sums are
// FP32; y is rounded once.
//
// Two forms of one kernel:
//   rows form (more than 128 tokens, larger products): the MMA's rows are tokens and its columns weight
//     rows, so a thread's scale is one number per block (its token's times its 128
//     columns').  A pair of CTAs (cta_group::2) computes 256 tokens x 256 weight rows, each
//     CTA loading 128 rows of either operand: 32 KB per block and SM instead of 48.
//     Persistent over tiles.
//   swapped form (up to 128 tokens, and small products): the MMA's 128 rows are weight rows and
//     its columns tokens, so a decode batch is not padded to 128 rows; scales vary over the
//     columns.  Bound by reading the weight.
// Measured, device time past L2 (M tokens, N x K weight):
//   4096, 13824 x 5120: 269 us, 2.16 PFLOP/s, in runs of tens of milliseconds (466 thousand clocks
//     at 1.6 to 1.75 GHz); 310 to 320 us, 1.8 to 1.9 PFLOP/s, in runs of seconds, which the power
//     limit holds at 1.4 to 1.5 GHz.  A block of 128 takes 846 clocks, of which its MMAs are 513; the
//     rest is the chain commit - read back - release of an accumulator.  A tile's beginning and end
//     are 5000 clocks, 13% of its time at 40 blocks.
//   512, 5120 x 5120: 23.4 us, 40 tiles on 74 pairs;  2048: 72 us, 160 tiles in three rounds
//   129, 5120 x 5120: 16.3 us, 20 tiles in three parts;  333, 1000 x 2064: 9.1 us (latency of one
//     chain of blocks)
//   1, 5120 x 5120: 8.6 us, 3.1 TB/s, 40 tiles in three parts of 13 and 14 blocks: starting up and
//     joining the parts weigh as much as the stream
//   16, 13824 x 5120: 15.2 us, 4.7 TB/s: 108 tiles, K not split, 40 SMs without work
// What was slower, where the kept form took 265 us at 4096 tokens: rows form with one accumulator
// pair of 256 columns (275 us at 4096 tokens, 29.0 at 512), without a pair of CTAs (128 x 256 tiles:
// 308), without moving registers (278), with eight promoting warps (279); swapped form with three
// smaller CTAs an SM (1 token 9.1 us, 16 tokens 17.1).
// The token scales come through a ring in shared memory that a warp of its own fills a few
// blocks ahead: loaded by the promoting warps themselves, one block ahead, their latency
// (about 1000 clocks under load) set the pace of the rows form.
//
// Where there are fewer tiles than CTA slots, a cluster of up to 8 CTAs splits K: each
// leaves its FP32 sums in its own shared memory and the cluster adds them in rank order
// over distributed shared memory, so the result does not depend on timing and no
// workspace or counter outlives the call.  CTA slots are what the device query counts: one
// CTA an SM, for the smaller tiles of the swapped form too, whatever their shared memory.
#include <algorithm>
#include <atomic>
#include <cmath>
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

// First device-side error of a stream's FP8 GEMMs, a word for each stream.  Word 0 is that of calls
// captured into graphs, which any stream may replay, and of streams that found no word left.
constexpr int kStatusWords = 1024;
__device__ int g_fp8_status[kStatusWords];

struct Fp8GemmParams {
  const float* xs;       // [KB][M]
  const float* ws;       // [NB][KB]
  void* y;
  int M, N, K, KB, NB;
  int tiles_a, tiles_b;  // tiles along the MMA's rows and columns
  int split;             // CTAs of the cluster that splits K
  int y_f32;
  int* status;           // the call's error word
  int drop;              // failure-path self test: the scales never arrive
  int vec;               // bytes of the widest aligned store of a y row: 32, 16, 8 or 2
};

// D(tmem) (+)= A(smem) * B(smem)^T, E4M3 operands, FP32 accumulation, K = 32; M = 128 in
// one CTA, or M = 256 over a pair (each CTA's 128 rows of A and half of B's rows).
template <bool kPair>
__device__ __forceinline__ void tc_mma_f8(uint32_t d_tmem, SmemDesc a, SmemDesc b, uint32_t idesc,
                                          uint32_t accumulate) {
  if constexpr (kPair)
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\t"
        "mov.b64 da, {%1, %2};\n\t"
        "mov.b64 db, {%3, %4};\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], da, db, %5, p;\n\t"
        "}" ::"r"(d_tmem),
        "r"(a.lo), "r"(a.hi), "r"(b.lo), "r"(b.hi), "r"(idesc), "r"(accumulate)
        : "memory");
  else
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

// Arrive on the barrier at this offset in every CTA of `mask` once the MMAs issued so far are done.
__device__ __forceinline__ void tc_commit_pair(uint32_t bar, uint16_t mask) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
      "h"(mask)
      : "memory");
}
__device__ __forceinline__ void tmem_alloc_pair(uint32_t dst_smem, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst_smem), "r"(ncols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc_pair(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}
// TMA load into this CTA's shared memory, counted on a barrier of either CTA of the pair.
__device__ __forceinline__ void tma_load_2d_pair(uint32_t dst, const CUtensorMap* m, uint32_t bar, int x, int y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(bar), "r"(x), "r"(y)
      : "memory");
}
// Arrive on a barrier of another CTA of the cluster (a mapa address).
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

// One lane of a converged warp.  The compiler knows that a branch on it leaves a single
// thread, so the operands of tcgen05 and TMA instructions go to uniform registers directly:
// four MMAs and two commits took about 300 clocks, after a branch on `lane == 0` 500.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
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
__device__ __forceinline__ float4 ld_dsmem4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr));
  return v;
}

template <bool kSwap, int kBN>
struct Cfg {
  static constexpr int kPair = kSwap ? 1 : 2;                  // CTAs of one MMA
  static constexpr int kGroups = !kSwap ? 4 : kBN >= 64 ? 2 : 1;            // promoting warpgroups
  static constexpr int kWarps = 4 * kGroups;                   // promoting warps
  static constexpr int kCols = kBN / kGroups;                  // columns per promoting thread
  static constexpr int kThreads = 128 + 128 * kGroups;
  static constexpr int kCtasPerSm = (kSwap && kBN <= 64) ? 2 : 1;
  static constexpr int kStageBytes = 16384 + (kSwap ? kBN * 128 : 16384);
  static constexpr int kStages = kSwap ? (kBN <= 16 ? 6 : kBN <= 32 ? 5 : kBN <= 64 ? 4 : 6) : 6;
  static constexpr int kSmem = kStages * kStageBytes + 1024;   // slack for the 1024-byte alignment
  // Accumulators in TMEM.  In the rows form each promoting warpgroup has its own 128
  // columns of the tile and two accumulators for them: with one accumulator pair of 256
  // columns, the chain multiply - read back - release set the pace (1200 clocks a block).
  static constexpr int kHalves = kSwap ? 1 : 2;
  static constexpr int kN = kBN / kHalves;                     // columns of one MMA
  static constexpr int kBufs = kSwap ? 4 : 2;
  static constexpr uint32_t kTmemCols = kBufs * kBN;
  static constexpr int kTok = kSwap ? kBN : 128;               // token scales per block
  static constexpr int kRing = kStages + kBufs;                // blocks of scales (see the scale warp)
  // Rows form: registers of a promoting thread and of the others.  They are moved by
  // setmaxnreg out of the block's launch allocation, which the three numbers have to fit.
  static constexpr int kRegLaunch = 96, kRegPromote = 104, kRegOther = 64;
  static constexpr int kRegTotal = 128 * kGroups * kRegPromote + 128 * kRegOther;
  static constexpr int kPitch = kSwap ? 128 : kBN + 4;         // floats per row of the split-K exchange
  static_assert(kStages * kStageBytes >= (kSwap ? kBN : 128) * kPitch * 4, "the exchange reuses the stages");
  static_assert(kSwap || kRegTotal <= kThreads * kRegLaunch, "more registers than the launch has");
  // a stage's "done" phase must be seen by the promoting warps before the next one ends
  static_assert(kBufs <= kStages && kTmemCols * kCtasPerSm <= 512, "");
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

// Stores four consecutive y values of one row (fewer at the row's end).
__device__ __forceinline__ void store4(const Fp8GemmParams& p, long long at, int n_left, const float* v) {
  if (p.y_f32 && p.vec >= 16) {
    *reinterpret_cast<float4*>(static_cast<float*>(p.y) + at) = make_float4(v[0], v[1], v[2], v[3]);
  } else if (!p.y_f32 && p.vec >= 8) {
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.y) + at) =
        make_uint2(bf16x2_from_f32(v[0], v[1]), bf16x2_from_f32(v[2], v[3]));
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (j < n_left) store_one(p, at + j, v[j]);
  }
}

template <bool kSwap, int kBN>
__global__ void __launch_bounds__(Cfg<kSwap, kBN>::kThreads, Cfg<kSwap, kBN>::kCtasPerSm)
fp8_gemm_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b,
                const Fp8GemmParams p) {
  using C = Cfg<kSwap, kBN>;
  constexpr bool kPair = C::kPair == 2;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t bars[(1 + C::kHalves) * C::kStages + C::kHalves * C::kBufs];
  __shared__ __align__(16) float ring[C::kRing][C::kTok + 4];
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_flag;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t smem = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t full0 = smem_u32(bars), done0 = full0 + 8 * C::kStages;
  const uint32_t tempty0 = done0 + 8 * C::kHalves * C::kStages;

  const int crank = kPair || p.split > 1 ? static_cast<int>(cluster_rank()) : 0;
  const int half = kPair ? crank & 1 : 0;              // which CTA of the pair
  if (warp == 0 && lane == 0) {
    prefetch_tmap(&tm_a);
    prefetch_tmap(&tm_b);
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(full0 + 8 * i, 1);
      for (int h = 0; h < C::kHalves; ++h) mbar_init(done0 + 8 * (h * C::kStages + i), 2);
    }
    for (int i = 0; i < C::kHalves * C::kBufs; ++i) mbar_init(tempty0 + 8 * i, C::kWarps / C::kHalves * C::kPair);
    abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    if (kPair) {
      tmem_alloc_pair(smem_u32(&tmem_slot), C::kTmemCols);
    } else {
      tmem_alloc(smem_u32(&tmem_slot), C::kTmemCols);
      tmem_relinquish();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (kPair) cluster_sync_all();                       // the pair's barriers exist
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(&tmem_slot);
  griddep_launch_dependents();

  // this CTA's tiles and its part of K
  const int part = crank / C::kPair, per = p.split * C::kPair;
  const int k0 = static_cast<int>(static_cast<long long>(p.KB) * part / p.split);
  const int k1 = static_cast<int>(static_cast<long long>(p.KB) * (part + 1) / p.split);
  const int first = static_cast<int>(blockIdx.x) / per, step = static_cast<int>(gridDim.x) / per;
  const int tiles = p.tiles_a * p.tiles_b;
  const uint32_t freed0 = done0 + 8 * (C::kHalves - 1) * C::kStages;   // of a block's last MMA
  volatile int* const stop = &abort_flag;
  auto give_up = [&] {
    *stop = 1;
    record_error(p.status, kDevErrTimeout);
  };

  // Rows form: the promoting warps take registers from the others.  Nobody takes any back
  // before the barrier that ends all roles: a warp without work that did so at once left the
  // promoting warps waiting for registers, and the block with them.
  if (warp < 4) {
    if (!kSwap) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kRegOther));
    if (warp == 0) {
      if (elect_one()) {
        // ---- producer.  The weight tiles of the first stages are requested before the wait
        // for the kernel before this one, which may be writing the activation.  A pair's
        // loads are all counted on the first CTA's barrier.
        auto load = [&](uint32_t dst, const CUtensorMap* m, int s, int kb, int row) {
          if (kPair) tma_load_2d_pair(dst, m, mapa(full0 + 8 * s, crank & ~1), kb * kFp8Block, row);
          else tma_load_2d(dst, m, full0 + 8 * s, kb * kFp8Block, row);
        };
        auto row_a = [&](int ta) { return kSwap ? ta * 128 : ta * 256 + half * 128; };
        // rows form: 64 rows of either half of the tile's 256, the other CTA has the next 64
        auto load_b = [&](uint32_t dst, int s, int kb, int tb) {
          if (kSwap) {
            load(dst, &tm_b, s, kb, tb * kBN);
          } else {
            load(dst, &tm_b, s, kb, tb * kBN + half * 64);
            load(dst + 8192, &tm_b, s, kb, tb * kBN + 128 + half * 64);
          }
        };
        int pre = 0;
        if (first < tiles) {
          int ta, tb;
          tile_at(first, p.tiles_a, p.tiles_b, ta, tb);
          for (; pre < C::kStages && k0 + pre < k1; ++pre) {
            const uint32_t st = smem + pre * C::kStageBytes;
            if (half == 0) mbar_arrive_expect_tx(full0 + 8 * pre, C::kStageBytes * C::kPair);
            if (kSwap) load(st, &tm_a, pre, k0 + pre, row_a(ta));
            else load_b(st + 16384, pre, k0 + pre, tb);
          }
        }
        griddep_wait();
        int it = 0, s = 0, phase = 1;
        bool ok = true;
        for (int t = first; ok && t < tiles; t += step) {
          int ta, tb;
          tile_at(t, p.tiles_a, p.tiles_b, ta, tb);
          for (int kb = k0; kb < k1; ++kb, ++it) {
            const uint32_t st = smem + s * C::kStageBytes;
            const bool done = it < pre;          // its weight tile is on the way
            if (it >= C::kStages && !mbar_wait(freed0 + 8 * s, phase, stop)) {
              ok = false;
              break;
            }
            if (!done && half == 0) mbar_arrive_expect_tx(full0 + 8 * s, C::kStageBytes * C::kPair);
            if (!(kSwap && done)) load(st, &tm_a, s, kb, row_a(ta));
            if (kSwap || !done) load_b(st + 16384, s, kb, tb);
            if (++s == C::kStages) {
              s = 0;
              phase ^= 1;
            }
          }
        }
        if (!ok) {
          // give up: wait (bounded) for the copies in flight before the memory is left
          give_up();
          const int zero = 0;
          if (half == 0)
            for (int j = max(0, it - C::kStages); j < it; ++j)
              mbar_wait(full0 + 8 * (j % C::kStages), (j / C::kStages) & 1, &zero);
        }
      }
    } else if (warp == 1) {
      if (half == 0 && elect_one()) {
        // ---- MMA issuer (the pair's first CTA).  It needs the activation, and its waits are
        // bounded: they begin when the kernel before this one has ended.
        griddep_wait();
        const uint32_t idesc =
            (1u << 4) | (static_cast<uint32_t>(C::kN >> 3) << 17) | (static_cast<uint32_t>(kPair ? 16 : 8) << 24);
        const SmemDesc a0 = make_sdesc(smem, 16, 1024, 2), b0 = make_sdesc(smem + 16384, 16, 1024, 2);
        int it = 0, s = 0, phase = 0, buf = 0, bphase = 1, issued = 0;
        bool ok = true;
        for (int t = first; ok && t < tiles; t += step) {
          for (int kb = k0; kb < k1; ++kb, ++it) {
            const uint32_t off = static_cast<uint32_t>(s) * (C::kStageBytes >> 4);
  #pragma unroll
            for (int h = 0; h < C::kHalves; ++h) {
              if ((h == 0 && !mbar_wait(full0 + 8 * s, phase, stop)) ||
                  (it >= C::kBufs && !mbar_wait(tempty0 + 8 * (h * C::kBufs + buf), bphase, stop))) {
                ok = false;
                break;
              }
              tc_fence_after();
  #pragma unroll
              for (int j = 0; j < 4; ++j)
                tc_mma_f8<kPair>(tmem + (h * C::kBufs + buf) * C::kN, sdesc_at(a0, off + 2 * j),
                                 sdesc_at(b0, off + h * (8192 >> 4) + 2 * j), idesc, j > 0);
              const uint32_t bar = done0 + 8 * (h * C::kStages + s);
              if (kPair) tc_commit_pair(bar, static_cast<uint16_t>(3u << (crank & ~1)));
              else tc_commit(bar);
              ++issued;
            }
            if (!ok) break;
            if (++s == C::kStages) {
              s = 0;
              phase ^= 1;
            }
            if (++buf == C::kBufs) {
              buf = 0;
              bphase ^= 1;
            }
          }
        }
        if (!ok) {
          give_up();
          // the products issued last, and so all before them, end before the tensor memory is freed
          // (bounded: where the barrier lacks its scales, the limit is long after their end)
          const int zero = 0, j = (issued - 1) / C::kHalves, h = (issued - 1) % C::kHalves;
          if (issued) mbar_wait(done0 + 8 * (h * C::kStages + j % C::kStages), (j / C::kStages) & 1, &zero);
        }
      }
    } else if (warp == 2) {
      // ---- scales: one ring slot per block, four blocks' loads in flight.  Swapped form:
      // each token's scale times the tile's weight scale; rows form: this CTA's 128 tokens'
      // scales, then the two weight scales of the tile's columns.  A block's "done" barriers
      // wait for its scales as well as for its MMAs, so block b may be filled in once block
      // b - kStages is done.  Its slot is then free too: the slot's last block, b - kStages -
      // kBufs, was read before the MMAs of block b - kStages were issued.
      griddep_wait();
      constexpr int kPer = (C::kTok + 31) / 32;
      int it = 0;
      bool ok = true;
      for (int t = p.drop ? tiles : first; ok && t < tiles; t += step) {
        int ta, tb;
        tile_at(t, p.tiles_a, p.tiles_b, ta, tb);
        const int tok0 = kSwap ? tb * kBN : ta * 256 + half * 128;
        const int wblk = kSwap ? ta : tb * 2 + (lane & 1);
        const float* pw = p.ws + static_cast<long long>(min(wblk, p.NB - 1)) * p.KB;
        for (int kb = k0; ok && kb < k1; kb += 4) {
          float s[4][kPer], w[4];
  #pragma unroll
          for (int q = 0; q < 4; ++q) {
            const bool in = kb + q < k1;
            w[q] = in ? __ldg(pw + kb + q) : 0.0f;
  #pragma unroll
            for (int j = 0; j < kPer; ++j) {
              const int m = tok0 + j * 32 + lane;
              const bool has = in && j * 32 + lane < C::kTok && m < p.M;
              s[q][j] = has ? __ldg(p.xs + static_cast<long long>(kb + q) * p.M + m) : 0.0f;
            }
          }
  #pragma unroll
          for (int q = 0; q < 4; ++q) {
            if (!ok || kb + q >= k1) break;
            const int slot = it % C::kRing, prev = it - C::kStages;
            const bool late =
                prev >= 0 && !mbar_wait(freed0 + 8 * (prev % C::kStages), (prev / C::kStages) & 1, stop);
            if (__any_sync(0xFFFFFFFFu, late)) {
              ok = false;
              break;
            }
  #pragma unroll
            for (int j = 0; j < kPer; ++j)
              if (j * 32 + lane < C::kTok) ring[slot][j * 32 + lane] = kSwap ? s[q][j] * w[q] : s[q][j];
            if (!kSwap && lane < 2) ring[slot][C::kTok + lane] = w[q];
            __syncwarp();
            if (lane < C::kHalves) mbar_arrive(done0 + 8 * (lane * C::kStages + it % C::kStages));
            ++it;
          }
        }
      }
      if (!ok) give_up();
    }
    __syncwarp();
  } else {
    // ---- promotion: one thread per MMA row and group of kCols columns
    if (!kSwap) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kRegPromote));
    griddep_wait();
    const int grp = (warp - 4) >> 2, row = (warp & 3) * 32 + lane;
    const int sub = kSwap ? 0 : grp >> 1;                     // rows form: this group's half of the tile
    const uint32_t taddr = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) +
                           (kSwap ? grp * C::kCols : sub * C::kBufs * C::kN + (grp & 1) * C::kCols);
    const uint32_t free0 = tempty0 + 8 * sub * C::kBufs, done_g = done0 + 8 * sub * C::kStages;
    const uint32_t release0 = kPair ? mapa(free0, crank & ~1) : free0;
    int s = 0, phase = 0, buf = 0, slot = 0;
    bool ok = true;
    // the next block's sums and scales are ready (all lanes of the warp agree)
    auto wait_block = [&] {
      if (!__all_sync(0xFFFFFFFFu, mbar_try_wait(done_g + 8 * s, phase)) &&
          __any_sync(0xFFFFFFFFu, !mbar_wait_slow(done_g + 8 * s, phase, stop))) {
        ok = false;
        give_up();
      }
      tc_fence_after();
      return ok;
    };
    auto release = [&] {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (kPair) mbar_arrive_cluster(release0 + 8 * buf);
        else mbar_arrive(release0 + 8 * buf);
      }
    };
    auto advance = [&] {
      if (++s == C::kStages) {
        s = 0;
        phase ^= 1;
      }
      if (++buf == C::kBufs) buf = 0;
      if (++slot == C::kRing) slot = 0;
    };
    for (int t = first; ok && t < tiles; t += step) {
      int ta, tb;
      tile_at(t, p.tiles_a, p.tiles_b, ta, tb);
      uint64_t acc[C::kCols / 2];
#pragma unroll
      for (int j = 0; j < C::kCols / 2; ++j) acc[j] = 0;
      if constexpr (kSwap) {
        for (int kb = k0; kb < k1; ++kb) {
          if (!wait_block()) break;
          // the scales are read before the accumulator (and with it their slot) is released
          const float* cs = &ring[slot][grp * C::kCols];
          const uint32_t src = taddr + buf * C::kN;
#pragma unroll
          for (int c = 0; c < C::kCols; c += 16) {
            uint64_t f[8];
#pragma unroll
            for (int j = 0; j < 8; j += 2) {
              const ulonglong2 q = *reinterpret_cast<const ulonglong2*>(cs + c + 2 * j);
              f[j] = q.x;
              f[j + 1] = q.y;
            }
            uint32_t d[16];
            tmem_ld16(src + c, d);
            if (c + 16 == C::kCols) release();
#pragma unroll
            for (int j = 0; j < 8; ++j)
              acc[c / 2 + j] = f32x2_fma(f32x2_pack(d[2 * j], d[2 * j + 1]), f[j], acc[c / 2 + j]);
          }
          advance();
        }
      } else {
        for (int kb = k0; kb < k1; ++kb) {
          if (!wait_block()) break;
          const uint32_t src = taddr + buf * C::kN;
          const float v = ring[slot][row] * ring[slot][C::kTok + sub];
          const uint64_t f = f32x2_pack(__float_as_uint(v), __float_as_uint(v));
#pragma unroll
          for (int c = 0; c < C::kCols; c += 16) {
            uint32_t d[16];
            tmem_ld16(src + c, d);
            if (c + 16 == C::kCols) release();
#pragma unroll
            for (int j = 0; j < 8; ++j)
              acc[c / 2 + j] = f32x2_fma(f32x2_pack(d[2 * j], d[2 * j + 1]), f, acc[c / 2 + j]);
          }
          advance();
        }
      }
      float v[C::kCols];
#pragma unroll
      for (int j = 0; j < C::kCols / 2; ++j)
        asm("mov.b64 {%0, %1}, %2;" : "=f"(v[2 * j]), "=f"(v[2 * j + 1]) : "l"(acc[j]));
      if (p.split > 1) {
        // The sums go into the stages, which every product of this CTA's part has to have read
        // first.  In the rows form a group has seen the end of its own half's products only; here they
        // meet, once, since a CTA that shares its tile has no other.  (A wait of the first half's groups
        // for the second half's barrier cost the loop above registers: 512 x 5120 x 5120 23.3 -> 24.7 us.)
        if (!kSwap) named_barrier(1, 128 * C::kGroups);
        float* x = reinterpret_cast<float*>(smem_raw + (smem - smem_u32(smem_raw)));
        if (!ok) {
          // products may still be under way: the stages stay as they are, y is not written
        } else if (kSwap) {
#pragma unroll
          for (int j = 0; j < C::kCols; ++j) x[(grp * C::kCols + j) * C::kPitch + row] = v[j];
        } else {
#pragma unroll
          for (int j = 0; j < C::kCols; j += 4)
            *reinterpret_cast<float4*>(x + row * C::kPitch + grp * C::kCols + j) =
                make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]);
        }
      } else if (ok) {
        if (kSwap) {
          const int n = ta * 128 + row, m = tb * kBN + grp * C::kCols;
          if (n < p.N) {
#pragma unroll
            for (int j = 0; j < C::kCols; ++j)
              if (m + j < p.M) store_one(p, static_cast<long long>(m + j) * p.N + n, v[j]);
          }
        } else {
          const int tok = ta * 256 + half * 128 + row, n = tb * kBN + grp * C::kCols;
          if (tok < p.M && n < p.N) store_row<C::kCols>(p, static_cast<long long>(tok) * p.N + n, p.N - n, v);
        }
      }
    }
    __syncwarp();
    if (!kSwap) {
      named_barrier(1, 128 * C::kGroups);      // between two setmaxnreg of a warpgroup
      asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kRegLaunch));
    }
  }

  // every role comes here, in the failing case too
  __syncthreads();
  if (!kSwap && warp < 4) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kRegLaunch));
  if (p.split > 1) {
    cluster_sync_all();
    // output rows of the exchange: tokens; this CTA finishes rows part, part + split, ...
    int ta, tb;
    tile_at(first, p.tiles_a, p.tiles_b, ta, tb);
    const int m0 = kSwap ? tb * kBN : ta * 256 + half * 128, n0 = kSwap ? ta * 128 : tb * kBN;
    constexpr int kRows = kSwap ? kBN : 128, kWide = kSwap ? 128 : kBN;
    const int rows = max(0, min(kRows, p.M - m0) - part);
    const bool good = *stop == 0;
    for (int i = tid; i < kWide / 4 * ((rows + p.split - 1) / p.split); i += C::kThreads) {
      const int c = i % (kWide / 4) * 4, r = part + i / (kWide / 4) * p.split;
      const uint32_t at = smem + (r * C::kPitch + c) * 4;
      float4 v[8 / C::kPair];                          // all parts' loads in flight, added in rank order
#pragma unroll
      for (int q = 0; q < 8 / C::kPair; ++q)
        v[q] = q < p.split ? ld_dsmem4(mapa(at, q * C::kPair + half)) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      float sum[4] = {v[0].x, v[0].y, v[0].z, v[0].w};
#pragma unroll
      for (int q = 1; q < 8 / C::kPair; ++q) {
        if (q >= p.split) break;
        sum[0] += v[q].x;
        sum[1] += v[q].y;
        sum[2] += v[q].z;
        sum[3] += v[q].w;
      }
      if (good && n0 + c < p.N) store4(p, static_cast<long long>(m0 + r) * p.N + n0 + c, p.N - n0 - c, sum);
    }
  }
  // nothing of a CTA that another one of the cluster reads or writes goes away early
  if (kPair || p.split > 1) cluster_sync_all();
  __syncwarp();
  if (warp == 1) {
    if (kPair) tmem_dealloc_pair(tmem, C::kTmemCols);
    else tmem_dealloc(tmem, C::kTmemCols);
  }
}

// What an instance needs to know about a device, found out on first use.
struct DeviceSetup {
  std::once_flag once;
  cudaError_t err = cudaSuccess;
  int* words = nullptr;        // the error words there
  int clusters[9] = {};        // clusters of 1..8 parts (pairs in the rows form) resident at once
};
constexpr int kMaxDevices = 64;

std::atomic<bool> g_drop_scales{false};   // failure-path self test, consumed by the next product

// The status words handed out on a device: word i is that of stream[i], i from 1 to `used`.  Fixed
// in size, since nothing may be thrown out of a C call.
struct StatusWords {
  cudaStream_t stream[kStatusWords];
  int used;
  bool shared;                           // word 0 may hold something
  int find(cudaStream_t s) const {
    int i = used;
    while (i > 0 && stream[i] != s) --i;
    return i;
  }
};
StatusWords g_words[kMaxDevices];
std::mutex g_words_mu;

// The word for a call on stream `s` of the current device `dev`; -1 where CUDA refuses.
int status_word(int dev, cudaStream_t s) {
  cudaStreamCaptureStatus capture;
  if (cudaStreamIsCapturing(s, &capture) != cudaSuccess) return -1;
  std::lock_guard<std::mutex> lk(g_words_mu);
  StatusWords& w = g_words[dev];
  if (capture == cudaStreamCaptureStatusNone) {
    const int at = w.find(s);
    if (at) return at;
    if (w.used + 1 < kStatusWords) {
      w.stream[++w.used] = s;
      return w.used;
    }
  }
  w.shared = true;
  return 0;
}

// Reads and clears a word on `s`.
int take_word(int word, cudaStream_t s) {
  int status = 0;
  if (cudaMemcpyFromSymbolAsync(&status, g_fp8_status, sizeof(int), word * sizeof(int), cudaMemcpyDeviceToHost, s) !=
          cudaSuccess ||
      cudaStreamSynchronize(s) != cudaSuccess)
    return BILOCO_ERR_CUDA;
  if (status != 0) {
    const int zero = 0;
    if (cudaMemcpyToSymbolAsync(g_fp8_status, &zero, sizeof(int), word * sizeof(int), cudaMemcpyHostToDevice, s) !=
            cudaSuccess ||
        cudaStreamSynchronize(s) != cudaSuccess)
      return BILOCO_ERR_CUDA;
  }
  return status;
}

template <bool kSwap, int kBN>
cudaError_t launch_instance(const CUtensorMap& ta, const CUtensorMap& tb, Fp8GemmParams& p, cudaStream_t s) {
  using C = Cfg<kSwap, kBN>;
  constexpr int kMaxSplit = 8 / C::kPair;
  static DeviceSetup setups[kMaxDevices];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= kMaxDevices) return cudaErrorInvalidDevice;
  DeviceSetup& d = setups[dev];
  auto kernel = fp8_gemm_kernel<kSwap, kBN>;
  std::call_once(d.once, [&] {
    d.err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (d.err != cudaSuccess) return;
    void* words = nullptr;
    d.err = cudaGetSymbolAddress(&words, g_fp8_status);
    if (d.err != cudaSuccess) return;
    d.words = static_cast<int*>(words);
    cudaFuncAttributes fa;
    d.err = cudaFuncGetAttributes(&fa, kernel);
    if (d.err != cudaSuccess) return;
    // with fewer registers at launch than are handed out the promoting warps would wait for ever
    if (!kSwap && fa.numRegs * C::kThreads < C::kRegTotal) {
      d.err = cudaErrorInvalidKernelImage;
      return;
    }
    for (int split = 1; split <= kMaxSplit; ++split) {
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3(static_cast<unsigned>(split * C::kPair));
      cfg.blockDim = dim3(C::kThreads);
      cfg.dynamicSmemBytes = C::kSmem;
      cudaLaunchAttribute attr;
      attr.id = cudaLaunchAttributeClusterDimension;
      attr.val.clusterDim.x = static_cast<unsigned>(split * C::kPair);
      attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
      cfg.attrs = &attr;
      cfg.numAttrs = 1;
      d.err = cudaOccupancyMaxActiveClusters(&d.clusters[split], kernel, &cfg);
      if (d.err != cudaSuccess) return;
    }
  });
  if (d.err != cudaSuccess) return d.err;
  const int word = status_word(dev, s);
  if (word < 0) return cudaErrorStreamCaptureImplicit;
  p.status = d.words + word;
  // K is split as far as all clusters still run at once, by the device's count (148 of one CTA, 74,
  // 45, 33, 26, 22, 15 and 15 of eight in the swapped form; 74 of one pair, 33, 22 and 15 in the rows
  // form): the weight's stream (or a tile's chain of blocks) gets shorter with every part, a second
  // wave costs more than it saves.  Measured, us at M, N, K (parts): 1, 5120, 5120: 13.3 (1), 8.6
  // (3); 129, 5120, 5120: 24.2 (1), 16.3 (3), 27.1 (4, does not fit).
  const long long tiles = static_cast<long long>(p.tiles_a) * p.tiles_b;
  int split = 1;
  for (int q = 2; q <= kMaxSplit && q <= p.KB; ++q)
    if (tiles <= d.clusters[q]) split = q;
  p.split = split;
  const long long slots = d.clusters[1];
  if (slots < 1) return cudaErrorCooperativeLaunchTooLarge;
  const unsigned groups = static_cast<unsigned>(split > 1 ? tiles * split : tiles < slots ? tiles : slots);
  return launch_pdl(kernel, groups * C::kPair, C::kThreads, C::kSmem, split * C::kPair, s, ta, tb, p);
}

}  // namespace

void fp8_drop_scales() { g_drop_scales.store(true); }

int fp8_take_status(cudaStream_t s) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return BILOCO_ERR_CUDA;
  if (dev >= kMaxDevices) return BILOCO_OK;
  int own = 0;
  bool shared = false;
  {
    std::lock_guard<std::mutex> lk(g_words_mu);
    own = g_words[dev].find(s);
    shared = g_words[dev].shared;
  }
  const int status = own ? take_word(own, s) : BILOCO_OK;
  if (status != BILOCO_OK || !shared) return status;
  // any stream's kernels may write word 0: wait for all of them, so that nothing is missed or cleared early
  if (cudaDeviceSynchronize() != cudaSuccess) return BILOCO_ERR_CUDA;
  return take_word(0, s);
}

// Columns of the swapped form's tiles.  Up to 32 tokens one tile takes all.  Above, small tiles
// give a small problem more CTAs, and parts of K; large ones read the weight fewer times.  The
// estimate, in units of one block's time in a tile of 128: the blocks of a CTA (as many as its SM
// holds share it) and 7 for the rest, of which a tile of up to 32 columns takes 0.6, and the
// operands of all tiles at 25 MB.  It is a fit to measured times, with two CTAs an SM up to 64
// columns; how K is split is decided by the device's count at the launch.  Measured, us with 32, 64, 128 columns: 5.3, 6.1, 7.9 (128 tokens,
// 512 x 2064), 7.6, 8.8, 9.3 (64, 2048 x 5120), 10.2, 10.0, 10.3 (128, 2048 x 5120), 15.5, 11.8, 12.6 (64,
// 5120 x 5120), 25.7, 21.1, 13.5 (128, 5120 x 5120), 15.9, 13.5, 10.7 (333, 1024 x 5120).
static int swapped_columns(int M, int NB, int KB) {
  if (M <= 32) return M <= 16 ? 16 : 32;
  const int sms = num_sms();
  int best = 0;
  double cost = 0.0;
  for (int bn = 32; bn <= 128; bn *= 2) {
    const double tiles = static_cast<double>(NB) * ((M + bn - 1) / bn), slots = bn <= 64 ? 2.0 * sms : sms;
    int split = 1;
    while (split < 8 && split < KB && tiles * (split + 1) <= slots) ++split;
    const double blocks = std::ceil(tiles / slots) * ((KB + split - 1) / split);
    const double shared = std::max(1.0, std::min(tiles * split, slots) / sms);
    const double c = (blocks * shared + 7.0) * (bn == 32 ? 0.6 : 1.0) + tiles * KB * (16384 + bn * 128) / 25e6;
    if (!best || c < cost) {
      best = bn;
      cost = c;
    }
  }
  return best;
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
  p.drop = g_drop_scales.exchange(false);
  const unsigned long long bits = reinterpret_cast<uintptr_t>(y) | static_cast<unsigned long long>(N) * (y_f32 ? 4 : 2);
  p.vec = bits % 32 == 0 ? 32 : bits % 16 == 0 ? 16 : bits % 8 == 0 ? 8 : 2;
  // Rows form above 128 tokens, except where a quarter of the SMs hold the swapped form's tiles,
  // so that four parts of K fit.  Across the borders, us at 5120 x 5120 and 1024 x 5120: 13.0 and 8.5
  // at 128 tokens (swapped), 15.7 at 129 (rows form, half of its 256 rows idle; swapped 23.0), 12.3
  // in the rows form and 9.6 swapped at 129; 2048 x 5120: 13.3 (rows) and 11.8 at 256 tokens, 32
  // tiles, 14.4 and 15.0 at 333, 48 tiles.
  const bool swap = M <= 128 || 4LL * p.NB * ((M + 127) / 128) <= num_sms();
  const int bn = swap ? swapped_columns(M, p.NB, p.KB) : 256;
  p.tiles_a = swap ? p.NB : (M + 255) / 256;
  p.tiles_b = swap ? (M + bn - 1) / bn : (N + bn - 1) / bn;
  if (static_cast<long long>(p.tiles_a) * p.tiles_b > 0x7FFFFFFFLL) return BILOCO_ERR_SHAPE;
  CUtensorMap tx, tw;
  if (!make_tmap(&tx, xq, K, M, swap ? bn : 128) || !make_tmap(&tw, wq, K, N, swap ? 128 : 64)) return BILOCO_ERR_CUDA;
  cudaError_t e;
  if (!swap) e = launch_instance<false, 256>(tx, tw, p, s);
  else if (bn == 16) e = launch_instance<true, 16>(tw, tx, p, s);
  else if (bn == 32) e = launch_instance<true, 32>(tw, tx, p, s);
  else if (bn == 64) e = launch_instance<true, 64>(tw, tx, p, s);
  else e = launch_instance<true, 128>(tw, tx, p, s);
  if (e == cudaErrorCooperativeLaunchTooLarge) return BILOCO_ERR_RESIDENCY;
  return e == cudaSuccess ? BILOCO_OK : BILOCO_ERR_CUDA;
}

}  // namespace biloco
