// vec.cuh -- 16-byte vector loads of bf16 rows and their conversion to fp32.
#pragma once

#include <cstdint>

namespace fp8mm {

// 16-byte streaming load (not kept in L1).  Coherent (no .nc): the kernels
// read inputs that the preceding kernel, overlapping them through
// programmatic dependent launch, may still be writing before their
// griddepcontrol.wait.
__device__ __forceinline__ uint4 ld_stream_16(const void* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

// The 8 bf16 values of a 16-byte vector as fp32 (exact).
__device__ __forceinline__ void bf16x8_to_f32(const uint4& v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

}  // namespace fp8mm
