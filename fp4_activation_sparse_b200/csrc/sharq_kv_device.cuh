// Device helpers shared by the attention kernels over the FP4 cache.
#pragma once

#include "sharq_common.cuh"

namespace sharq {

__device__ __forceinline__ uint32_t kv_smem_u32(const void *p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }
__device__ __forceinline__ float kv_ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t mul2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t kv_pack_half2(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}
__device__ __forceinline__ void sts128(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
// two scale codes in the low 16 bits -> half2 (low byte in the low half): exact in the cache's
// range of exponents
template <bool MX>
__device__ __forceinline__ uint32_t kv_scales2(uint32_t two) {
  uint32_t d;
  if (MX) {
    d = kv_pack_half2(__uint_as_float((two & 0xFFu) << 23), __uint_as_float((two & 0xFF00u) << 15));
  } else {
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(d) : "h"((uint16_t)two));
  }
  return d;
}

}  // namespace sharq
