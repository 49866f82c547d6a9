// Promotion of a block's sums out of tensor memory: 32 columns of FP32 block sums times
// their scales, added to running sums held as pairs (fma.rn.f32x2).
//
// tcgen05.ld fills its registers asynchronously, so the load of the next 32 columns, the
// 16 packed FMAs on the current ones and the wait for the load are one asm statement: the
// load's latency passes behind the FMAs, and no instruction of the compiler's can touch
// the registers before they are filled.
#pragma once

#include <cstdint>

#include "ptx.cuh"

namespace biloco {

__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&v)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
        "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]), "=r"(v[16]),
        "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]),
        "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
      : "r"(taddr)
      : "memory");
}

// acc += cur * s for 32 columns while the next 32 are loaded into nx.
__device__ __forceinline__ void promote32_ld(uint64_t* acc, const uint32_t (&cur)[32], uint64_t s, uint32_t taddr,
                                             uint32_t (&nx)[32]) {
  asm volatile(
      "{\n\t.reg .b64 t;\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%48];\n\t"
      "mov.b64 t, {%49,%50}; fma.rn.f32x2 %32, t, %81, %32;\n\t"
      "mov.b64 t, {%51,%52}; fma.rn.f32x2 %33, t, %81, %33;\n\t"
      "mov.b64 t, {%53,%54}; fma.rn.f32x2 %34, t, %81, %34;\n\t"
      "mov.b64 t, {%55,%56}; fma.rn.f32x2 %35, t, %81, %35;\n\t"
      "mov.b64 t, {%57,%58}; fma.rn.f32x2 %36, t, %81, %36;\n\t"
      "mov.b64 t, {%59,%60}; fma.rn.f32x2 %37, t, %81, %37;\n\t"
      "mov.b64 t, {%61,%62}; fma.rn.f32x2 %38, t, %81, %38;\n\t"
      "mov.b64 t, {%63,%64}; fma.rn.f32x2 %39, t, %81, %39;\n\t"
      "mov.b64 t, {%65,%66}; fma.rn.f32x2 %40, t, %81, %40;\n\t"
      "mov.b64 t, {%67,%68}; fma.rn.f32x2 %41, t, %81, %41;\n\t"
      "mov.b64 t, {%69,%70}; fma.rn.f32x2 %42, t, %81, %42;\n\t"
      "mov.b64 t, {%71,%72}; fma.rn.f32x2 %43, t, %81, %43;\n\t"
      "mov.b64 t, {%73,%74}; fma.rn.f32x2 %44, t, %81, %44;\n\t"
      "mov.b64 t, {%75,%76}; fma.rn.f32x2 %45, t, %81, %45;\n\t"
      "mov.b64 t, {%77,%78}; fma.rn.f32x2 %46, t, %81, %46;\n\t"
      "mov.b64 t, {%79,%80}; fma.rn.f32x2 %47, t, %81, %47;\n\t"
      "tcgen05.wait::ld.sync.aligned;\n\t}"
      : "=&r"(nx[0]), "=&r"(nx[1]), "=&r"(nx[2]), "=&r"(nx[3]), "=&r"(nx[4]), "=&r"(nx[5]), "=&r"(nx[6]),
        "=&r"(nx[7]), "=&r"(nx[8]), "=&r"(nx[9]), "=&r"(nx[10]), "=&r"(nx[11]), "=&r"(nx[12]), "=&r"(nx[13]),
        "=&r"(nx[14]), "=&r"(nx[15]), "=&r"(nx[16]), "=&r"(nx[17]), "=&r"(nx[18]), "=&r"(nx[19]), "=&r"(nx[20]),
        "=&r"(nx[21]), "=&r"(nx[22]), "=&r"(nx[23]), "=&r"(nx[24]), "=&r"(nx[25]), "=&r"(nx[26]), "=&r"(nx[27]),
        "=&r"(nx[28]), "=&r"(nx[29]), "=&r"(nx[30]), "=&r"(nx[31]), "+l"(acc[0]), "+l"(acc[1]), "+l"(acc[2]),
        "+l"(acc[3]), "+l"(acc[4]), "+l"(acc[5]), "+l"(acc[6]), "+l"(acc[7]), "+l"(acc[8]), "+l"(acc[9]),
        "+l"(acc[10]), "+l"(acc[11]), "+l"(acc[12]), "+l"(acc[13]), "+l"(acc[14]), "+l"(acc[15])
      : "r"(taddr), "r"(cur[0]), "r"(cur[1]), "r"(cur[2]), "r"(cur[3]), "r"(cur[4]), "r"(cur[5]), "r"(cur[6]),
        "r"(cur[7]), "r"(cur[8]), "r"(cur[9]), "r"(cur[10]), "r"(cur[11]), "r"(cur[12]), "r"(cur[13]), "r"(cur[14]),
        "r"(cur[15]), "r"(cur[16]), "r"(cur[17]), "r"(cur[18]), "r"(cur[19]), "r"(cur[20]), "r"(cur[21]),
        "r"(cur[22]), "r"(cur[23]), "r"(cur[24]), "r"(cur[25]), "r"(cur[26]), "r"(cur[27]), "r"(cur[28]),
        "r"(cur[29]), "r"(cur[30]), "r"(cur[31]), "l"(s)
      : "memory");
}
// The same with a scale per column (16 pairs).
__device__ __forceinline__ void promote32_ld(uint64_t* acc, const uint32_t (&cur)[32], const uint64_t (&s)[16],
                                             uint32_t taddr, uint32_t (&nx)[32]) {
  asm volatile(
      "{\n\t.reg .b64 t;\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%48];\n\t"
      "mov.b64 t, {%49,%50}; fma.rn.f32x2 %32, t, %81, %32;\n\t"
      "mov.b64 t, {%51,%52}; fma.rn.f32x2 %33, t, %82, %33;\n\t"
      "mov.b64 t, {%53,%54}; fma.rn.f32x2 %34, t, %83, %34;\n\t"
      "mov.b64 t, {%55,%56}; fma.rn.f32x2 %35, t, %84, %35;\n\t"
      "mov.b64 t, {%57,%58}; fma.rn.f32x2 %36, t, %85, %36;\n\t"
      "mov.b64 t, {%59,%60}; fma.rn.f32x2 %37, t, %86, %37;\n\t"
      "mov.b64 t, {%61,%62}; fma.rn.f32x2 %38, t, %87, %38;\n\t"
      "mov.b64 t, {%63,%64}; fma.rn.f32x2 %39, t, %88, %39;\n\t"
      "mov.b64 t, {%65,%66}; fma.rn.f32x2 %40, t, %89, %40;\n\t"
      "mov.b64 t, {%67,%68}; fma.rn.f32x2 %41, t, %90, %41;\n\t"
      "mov.b64 t, {%69,%70}; fma.rn.f32x2 %42, t, %91, %42;\n\t"
      "mov.b64 t, {%71,%72}; fma.rn.f32x2 %43, t, %92, %43;\n\t"
      "mov.b64 t, {%73,%74}; fma.rn.f32x2 %44, t, %93, %44;\n\t"
      "mov.b64 t, {%75,%76}; fma.rn.f32x2 %45, t, %94, %45;\n\t"
      "mov.b64 t, {%77,%78}; fma.rn.f32x2 %46, t, %95, %46;\n\t"
      "mov.b64 t, {%79,%80}; fma.rn.f32x2 %47, t, %96, %47;\n\t"
      "tcgen05.wait::ld.sync.aligned;\n\t}"
      : "=&r"(nx[0]), "=&r"(nx[1]), "=&r"(nx[2]), "=&r"(nx[3]), "=&r"(nx[4]), "=&r"(nx[5]), "=&r"(nx[6]),
        "=&r"(nx[7]), "=&r"(nx[8]), "=&r"(nx[9]), "=&r"(nx[10]), "=&r"(nx[11]), "=&r"(nx[12]), "=&r"(nx[13]),
        "=&r"(nx[14]), "=&r"(nx[15]), "=&r"(nx[16]), "=&r"(nx[17]), "=&r"(nx[18]), "=&r"(nx[19]), "=&r"(nx[20]),
        "=&r"(nx[21]), "=&r"(nx[22]), "=&r"(nx[23]), "=&r"(nx[24]), "=&r"(nx[25]), "=&r"(nx[26]), "=&r"(nx[27]),
        "=&r"(nx[28]), "=&r"(nx[29]), "=&r"(nx[30]), "=&r"(nx[31]), "+l"(acc[0]), "+l"(acc[1]), "+l"(acc[2]),
        "+l"(acc[3]), "+l"(acc[4]), "+l"(acc[5]), "+l"(acc[6]), "+l"(acc[7]), "+l"(acc[8]), "+l"(acc[9]),
        "+l"(acc[10]), "+l"(acc[11]), "+l"(acc[12]), "+l"(acc[13]), "+l"(acc[14]), "+l"(acc[15])
      : "r"(taddr), "r"(cur[0]), "r"(cur[1]), "r"(cur[2]), "r"(cur[3]), "r"(cur[4]), "r"(cur[5]), "r"(cur[6]),
        "r"(cur[7]), "r"(cur[8]), "r"(cur[9]), "r"(cur[10]), "r"(cur[11]), "r"(cur[12]), "r"(cur[13]), "r"(cur[14]),
        "r"(cur[15]), "r"(cur[16]), "r"(cur[17]), "r"(cur[18]), "r"(cur[19]), "r"(cur[20]), "r"(cur[21]),
        "r"(cur[22]), "r"(cur[23]), "r"(cur[24]), "r"(cur[25]), "r"(cur[26]), "r"(cur[27]), "r"(cur[28]),
        "r"(cur[29]), "r"(cur[30]), "r"(cur[31]), "l"(s[0]), "l"(s[1]), "l"(s[2]), "l"(s[3]), "l"(s[4]), "l"(s[5]),
        "l"(s[6]), "l"(s[7]), "l"(s[8]), "l"(s[9]), "l"(s[10]), "l"(s[11]), "l"(s[12]), "l"(s[13]), "l"(s[14]),
        "l"(s[15])
      : "memory");
}

// acc += cur * s without a further load.
__device__ __forceinline__ void promote32(uint64_t* acc, const uint32_t (&cur)[32], uint64_t s) {
#pragma unroll
  for (int j = 0; j < 16; ++j) acc[j] = f32x2_fma(f32x2_pack(cur[2 * j], cur[2 * j + 1]), s, acc[j]);
}
__device__ __forceinline__ void promote32(uint64_t* acc, const uint32_t (&cur)[32], const uint64_t (&s)[16]) {
#pragma unroll
  for (int j = 0; j < 16; ++j) acc[j] = f32x2_fma(f32x2_pack(cur[2 * j], cur[2 * j + 1]), s[j], acc[j]);
}

}  // namespace biloco
