// gda_prefill_dev.cuh -- device helpers that the persistent prompt kernels share (sm_103a): a
// suspended barrier poll and the gate's sigmoid.
#pragma once

#include "gda_tc.cuh"

namespace gda {

// One poll of a barrier, suspended up to about `ns`.
__device__ __forceinline__ bool mbar_try_wait_for(uint64_t* bar, uint32_t parity, uint32_t ns) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity), "r"(ns)
      : "memory");
  return ok != 0;
}

__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ __nv_bfloat162 bits_bf162(uint32_t u) {
  return __halves2bfloat162(__ushort_as_bfloat16((unsigned short)u), __ushort_as_bfloat16((unsigned short)(u >> 16)));
}
// the sigmoids of 8 gates from the table of all 65536 (rarely needed, out of line)
static __device__ __noinline__ uint4 table_sigmoids(uint4 g, const uint16_t* table) {
  uint32_t v[4] = {g.x, g.y, g.z, g.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) v[e] = __ldg(table + (v[e] & 0xFFFFu)) | ((uint32_t)__ldg(table + (v[e] >> 16)) << 16);
  return make_uint4(v[0], v[1], v[2], v[3]);
}
// 4 R pairs of BF16 gates become RNE_bf16(sigmoid), without a branch between them, so that
// their chains of SFU operations overlap.  A BF16 gate has 65536 values, so the approximation
// is judged by all of them: 1 / (1 + 2^(-g log2 e)) with the approximate exponential and
// reciprocal rounds to the correct BF16 value for every g >= -87 (also with the constant one
// step lower or two higher).  Below that the exponential leaves the reciprocal's range, whose
// results would be subnormal: such gates and NaNs come from the table.
template <int R>
__device__ __forceinline__ void sigmoids(uint32_t* g, const uint16_t* table) {
  constexpr float kNegLog2e = -1.4426950408889634f, kLowest = -87.0f;
  uint32_t sg[4 * R];
  __nv_bfloat162 least = bits_bf162(g[0]);
#pragma unroll
  for (int e = 0; e < 4 * R; ++e) {
    if (e > 0) least = __hmin2_nan(least, bits_bf162(g[e]));
    const float2 x = mul_f32x2(make_float2(__uint_as_float(g[e] << 16), __uint_as_float(g[e] & 0xFFFF0000u)),
                               make_float2(kNegLog2e, kNegLog2e));
    const float2 d = add_f32x2(make_float2(ex2_approx(x.x), ex2_approx(x.y)), make_float2(1.0f, 1.0f));
    sg[e] = bf16x2_rn(rcp_approx(d.x), rcp_approx(d.y));
  }
  if (!(__low2float(least) >= kLowest && __high2float(least) >= kLowest)) {
#pragma unroll
    for (int y = 0; y < R; ++y) {
      const uint4 v = table_sigmoids(make_uint4(g[4 * y], g[4 * y + 1], g[4 * y + 2], g[4 * y + 3]), table);
      sg[4 * y] = v.x, sg[4 * y + 1] = v.y, sg[4 * y + 2] = v.z, sg[4 * y + 3] = v.w;
    }
  }
#pragma unroll
  for (int e = 0; e < 4 * R; ++e) g[e] = sg[e];
}

}  // namespace gda
