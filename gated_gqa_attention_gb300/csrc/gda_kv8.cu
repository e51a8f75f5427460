// gda_kv8.cu -- writing rows into the 8-bit (e4m3) KV cache and reading them back as BF16.
//
// kv8_write: code = nearest e4m3 to x / descale (ties to even, beyond 448 to 448), the quotient
//   one FP32 IEEE division.  512 bytes in, 256 out per row.
// kv8_gather: RNE_bf16(descale * e4m3(code)), the product one FP32 rounding: the rows that
//   indices name, packed, as a prompt's attention reads them (prefill_packed).
// A warp takes one (token, KV head), K and V rows together; lane l owns dimensions 8l .. 8l + 7
// (16 bytes of BF16, 8 of codes), so every load and store of the warp is one contiguous row.  With
// two units a warp 16384 tokens x 2 heads (written, then read) take 21.6 us, with four 23.5.
//
// Divisions would bound the write (20.6 us for both kernels of that call), so the codes come from
// products with the reciprocal r where they must be the same.  r and y = x r are each rounded once,
// so y is within 2^-22 of x / descale, and so is the IEEE quotient; rounding to e4m3 is monotone, so
// where y (1 - 2^-21) and y (1 + 2^-21) have the same code it is the quotient's.  Otherwise (next to
// a border between codes) the lane's eight values are divided.  (A product that leaves FP32's
// normal range below or above is far below 2^-10 or above 464, where every code is 0 or 448.)
// Powers of two have exact reciprocals and need no test; a descale whose reciprocal is not a normal
// number is divided by.  The floor is HBM's: 16384 tokens x 2 heads 14.9 us.
#include "gda_kernels.h"
#include "gda_kv4.cuh"
#include "gda_tc.cuh"

namespace gda {

namespace {

__device__ __forceinline__ uint32_t e4m3x2_rn(float lo, float hi) {
  uint32_t r;
  asm("{\n\t.reg .b16 t;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 t, %1, %2;\n\t"
      "mov.b32 %0, {t, 0};\n\t}"
      : "=r"(r)
      : "f"(hi), "f"(lo));
  return r;
}

// eight BF16 values as codes
__device__ __forceinline__ uint2 codes_of(const uint4& v, const Kv8Factor& d) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t c[4], differ = d.mode == kKv8Divide ? 1u : 0u;
  if (d.mode != kKv8Divide) {
    const float2 r = make_float2(d.reciprocal, d.reciprocal);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 y = mul_f32x2(make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u)), r);
      if (d.mode == kKv8Exact) {
        c[i] = e4m3x2_rn(y.x, y.y);
      } else {
        constexpr float kBelow = 1.0f - 4.76837158203125e-7f, kAbove = 1.0f + 4.76837158203125e-7f;  // 1 -+ 2^-21
        const float2 lo = mul_f32x2(y, make_float2(kBelow, kBelow)), hi = mul_f32x2(y, make_float2(kAbove, kAbove));
        c[i] = e4m3x2_rn(lo.x, lo.y);
        differ |= c[i] ^ e4m3x2_rn(hi.x, hi.y);
      }
    }
  }
  if (differ != 0u) {
#pragma unroll 1
    for (int i = 0; i < 8; ++i) {  // (rolled: rarely run)
      const uint32_t word = i < 2 ? v.x : i < 4 ? v.y : i < 6 ? v.z : v.w;
      const float x = __uint_as_float((i & 1) ? word & 0xFFFF0000u : word << 16);
      const uint32_t code = (e4m3x2_rn(__fdiv_rn(x, d.descale), 0.0f) & 0xFFu) << (8 * (i & 1));
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (k == i >> 1) c[k] = (i & 1) ? c[k] | code : code;
    }
  }
  return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}
__device__ __forceinline__ uint4 bf16_of(const uint2& c, float descale) {
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t f = e4m3x2_to_f16x2((i < 2 ? c.x : c.y) >> (16 * (i & 1)));
    const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&f));
    o[i] = pack_bf16x2(descale * v.x, descale * v.y);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

__global__ void __launch_bounds__(256) kv8_write_kernel(const __grid_constant__ Kv8WriteParams p) {
  const long long w = ((long long)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  const int lane = threadIdx.x & 31;
  pdl_wait_prior_grid();
  pdl_launch_dependents();
  if (w >= p.T * p.Hkv) return;  // whole warps
  const long long t = w / p.Hkv;
  const int h = (int)(w - t * p.Hkv);
  const uint4 rk = __ldcs(reinterpret_cast<const uint4*>(p.k + t * p.k_stride + (long long)h * kD) + lane);
  const uint4 rv = __ldcs(reinterpret_cast<const uint4*>(p.v + t * p.v_stride + (long long)h * kD) + lane);
  const int slot = __ldg(p.slots + t);
  if (slot < 0 || (long long)slot >= p.num_slots) return;
  const size_t row = ((size_t)slot * p.Hkv + h) * kD;
  reinterpret_cast<uint2*>(p.k_pool + row)[lane] = codes_of(rk, p.k_factor);
  reinterpret_cast<uint2*>(p.v_pool + row)[lane] = codes_of(rv, p.v_factor);
}

__global__ void __launch_bounds__(256) kv8_gather_kernel(const __grid_constant__ Kv8GatherParams p) {
  const long long w = ((long long)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  const int lane = threadIdx.x & 31;
  pdl_wait_prior_grid();
  pdl_launch_dependents();
  if (w >= p.N * p.Hkv) return;  // whole warps
  const long long i = w / p.Hkv;
  const int h = (int)(w - i * p.Hkv);
  const int slot = __ldg(p.indices + i);
  uint2 ck = make_uint2(0u, 0u), cv = ck;   // an index outside the pools reads zeros
  if (slot >= 0 && (long long)slot < p.num_slots) {
    const size_t row = ((size_t)slot * p.Hkv + h) * kD;
    ck = __ldcs(reinterpret_cast<const uint2*>(p.k_pool + row) + lane);
    cv = __ldcs(reinterpret_cast<const uint2*>(p.v_pool + row) + lane);
  }
  reinterpret_cast<uint4*>(p.k_out + w * kD)[lane] = bf16_of(ck, p.k_descale);
  reinterpret_cast<uint4*>(p.v_out + w * kD)[lane] = bf16_of(cv, p.v_descale);
}

// As a programmatic dependent: a read that follows a write (or the next step's write) is launched
// during its end.
template <typename P>
cudaError_t launch8(void (*kernel)(P), const P& p, long long units, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((units + 7) / 8));
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

}  // namespace

cudaError_t launch_kv8_write(const Kv8WriteParams& p, cudaStream_t stream) {
  return launch8(kv8_write_kernel, p, p.T * p.Hkv, stream);
}

cudaError_t launch_kv8_gather(const Kv8GatherParams& p, cudaStream_t stream) {
  return launch8(kv8_gather_kernel, p, p.N * p.Hkv, stream);
}

}  // namespace gda
