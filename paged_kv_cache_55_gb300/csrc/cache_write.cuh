// Helpers of the kernels that write rows into the paged cache (sm_103a):
// the E4M3 quantisers and the rotary table load.
#pragma once

#include "pa_common.cuh"

namespace pa {

// 8-bit caches (LLM-infra reading map, §4.2: the cache is quantised online
// as it is written): the same slots, each element stored as the E4M3 code of
// its binary32 quotient by the cache's scale. One thread turns 16 elements
// (two 16-byte loads) into one 16-byte vector of codes.
template <typename E>
__device__ __forceinline__ uint4 quantize16(uint4 a, uint4 b, float scale) {
  const uint32_t x[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  uint32_t c[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint32_t p0 = e4m3x2_from_f32(__fdiv_rn(E::lo(x[2 * k]), scale), __fdiv_rn(E::hi(x[2 * k]), scale));
    const uint32_t p1 =
        e4m3x2_from_f32(__fdiv_rn(E::lo(x[2 * k + 1]), scale), __fdiv_rn(E::hi(x[2 * k + 1]), scale));
    c[k] = p0 | (p1 << 16);
  }
  return make_uint4(c[0], c[1], c[2], c[3]);
}

// Eight elements -> eight E4M3 codes of x / scale (the quantiser of reshape_and_cache_fp8).
template <typename E>
__device__ __forceinline__ uint2 quantize8(uint4 a, float scale) {
  const uint32_t x[4] = {a.x, a.y, a.z, a.w};
  uint32_t c[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const uint32_t p0 = e4m3x2_from_f32(__fdiv_rn(E::lo(x[2 * k]), scale), __fdiv_rn(E::hi(x[2 * k]), scale));
    const uint32_t p1 =
        e4m3x2_from_f32(__fdiv_rn(E::lo(x[2 * k + 1]), scale), __fdiv_rn(E::hi(x[2 * k + 1]), scale));
    c[k] = p0 | (p1 << 16);
  }
  return make_uint2(c[0], c[1]);
}

// Four floats of a table written before this kernel (the rotary table may come
// from an earlier kernel of the stream): a volatile, L1-cached load that the
// compiler cannot hoist above griddep_wait (as it may an invariant load).
__device__ __forceinline__ float4 ld_ca4(const float *p) {
  float4 v;
  asm volatile("ld.global.ca.v4.f32 {%0, %1, %2, %3}, [%4];\n"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "l"(p)
               : "memory");
  return v;
}

}  // namespace pa
