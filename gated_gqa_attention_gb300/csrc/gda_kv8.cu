// gda_kv8.cu -- writing rows into the 8-bit (e4m3) KV cache and reading them back as BF16.
//
// kv8_write: code = nearest e4m3 to x / descale (ties to even, beyond 448 to 448), the quotient
//   one FP32 IEEE division, or an exact product where both descales are powers of two.
//   512 bytes in, 256 out per row: bound by HBM for a prompt, by the launch for a decode step.
// kv8_gather: RNE_bf16(descale * e4m3(code)), the product one FP32 rounding: the rows that
//   indices name, packed, as a prompt's attention reads them (prefill_packed).
// A warp takes (token, KV head) units, K and V rows together; lane l owns dimensions 8l .. 8l + 7
// (16 bytes of BF16, 8 of codes), so every load and store of the warp is one contiguous row.
#include "gda_kernels.h"
#include "gda_kv4.cuh"

namespace gda {

namespace {

constexpr int kUnits8 = 2;   // units a warp has in flight

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
template <bool kInv>
__device__ __forceinline__ uint2 codes_of(const uint4& v, float factor) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float lo = __uint_as_float(w[i] << 16), hi = __uint_as_float(w[i] & 0xFFFF0000u);
    c[i] = kInv ? e4m3x2_rn(lo * factor, hi * factor) : e4m3x2_rn(__fdiv_rn(lo, factor), __fdiv_rn(hi, factor));
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

template <bool kInv>
__global__ void __launch_bounds__(256) kv8_write_kernel(const __grid_constant__ Kv8WriteParams p) {
  const long long n = p.T * p.Hkv;
  const long long w0 = (((long long)blockIdx.x * blockDim.x + threadIdx.x) >> 5) * kUnits8;
  const int lane = threadIdx.x & 31;
  uint4 rk[kUnits8], rv[kUnits8];
  long long row[kUnits8];   // cache row, -1: not written
#pragma unroll
  for (int u = 0; u < kUnits8; ++u) {
    const long long w = w0 + u;
    row[u] = -1;
    if (w >= n) continue;   // (the same for the whole warp)
    const long long t = w / p.Hkv;
    const int h = (int)(w - t * p.Hkv);
    rk[u] = __ldcs(reinterpret_cast<const uint4*>(p.k + t * p.k_stride + (long long)h * kD) + lane);
    rv[u] = __ldcs(reinterpret_cast<const uint4*>(p.v + t * p.v_stride + (long long)h * kD) + lane);
    const int slot = __ldg(p.slots + t);
    if (slot >= 0 && (long long)slot < p.num_slots) row[u] = (long long)slot * p.Hkv + h;
  }
#pragma unroll
  for (int u = 0; u < kUnits8; ++u) {
    if (row[u] < 0) continue;
    reinterpret_cast<uint2*>(p.k_pool + row[u] * kD)[lane] = codes_of<kInv>(rk[u], p.k_factor);
    reinterpret_cast<uint2*>(p.v_pool + row[u] * kD)[lane] = codes_of<kInv>(rv[u], p.v_factor);
  }
}

__global__ void __launch_bounds__(256) kv8_gather_kernel(const __grid_constant__ Kv8GatherParams p) {
  const long long n = p.N * p.Hkv;
  const long long w0 = (((long long)blockIdx.x * blockDim.x + threadIdx.x) >> 5) * kUnits8;
  const int lane = threadIdx.x & 31;
  uint2 ck[kUnits8], cv[kUnits8];
#pragma unroll
  for (int u = 0; u < kUnits8; ++u) {
    const long long w = w0 + u;
    ck[u] = cv[u] = make_uint2(0u, 0u);   // an index outside the pools reads zeros
    if (w >= n) continue;
    const long long i = w / p.Hkv;
    const int h = (int)(w - i * p.Hkv);
    const int slot = __ldg(p.indices + i);
    if (slot >= 0 && (long long)slot < p.num_slots) {
      const size_t row = (size_t)slot * p.Hkv + h;
      ck[u] = __ldcs(reinterpret_cast<const uint2*>(p.k_pool + row * kD) + lane);
      cv[u] = __ldcs(reinterpret_cast<const uint2*>(p.v_pool + row * kD) + lane);
    }
  }
#pragma unroll
  for (int u = 0; u < kUnits8; ++u) {
    const long long w = w0 + u;
    if (w >= n) continue;
    reinterpret_cast<uint4*>(p.k_out + w * kD)[lane] = bf16_of(ck[u], p.k_descale);
    reinterpret_cast<uint4*>(p.v_out + w * kD)[lane] = bf16_of(cv[u], p.v_descale);
  }
}

unsigned blocks_for(long long units) { return (unsigned)((units + 8 * kUnits8 - 1) / (8 * kUnits8)); }

}  // namespace

cudaError_t launch_kv8_write(const Kv8WriteParams& p, cudaStream_t stream) {
  const unsigned blocks = blocks_for(p.T * p.Hkv);
  if (p.inv) kv8_write_kernel<true><<<blocks, 256, 0, stream>>>(p);
  else kv8_write_kernel<false><<<blocks, 256, 0, stream>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_kv8_gather(const Kv8GatherParams& p, cudaStream_t stream) {
  kv8_gather_kernel<<<blocks_for(p.N * p.Hkv), 256, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace gda
