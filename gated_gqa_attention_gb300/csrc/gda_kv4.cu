// gda_kv4.cu -- writing rows into the 4-bit KV cache and reading them back as BF16.
//
// kv4_write: the K and V rows of T tokens, quantised (gda_kv4.cuh) into their slots.
//   Reads 1024 bytes and writes 288 per (token, KV head): bound by HBM for a prompt, by
//   the launch for a decode step.
// kv4_gather: the rows that N indices name, as packed BF16 tensors -- what the prompt
//   attention reads when a prompt continues after a prefix held in the cache.
//   value = RNE_bf16(descale * (e4m3(scale) * e2m1(code))), the product of scale and
//   code exact, the descale one FP32 rounding.  288 bytes in, 1024 out.
// One warp per (token, KV head), K and V together: lane l owns dimensions 8l .. 8l + 7
// (16 bytes of BF16, 4 bytes of codes), so every load and store of the warp is one
// contiguous row and both rows are in flight at a time.
#include "gda_kernels.h"
#include "gda_kv4.cuh"

namespace gda {

namespace {

__device__ __forceinline__ void bf16x8_to_float(const uint4& r, float* f) {
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

// dimensions 8 lane .. + 7 of a row: codes c, their block's scale code
__device__ __forceinline__ uint4 row4_to_bf16(uint32_t c, uint32_t scale, float descale) {
  const float s = __half2float(__ushort_as_half((unsigned short)(e4m3x2_to_f16x2(scale) & 0xFFFFu)));
  uint32_t f[4], o[4];
  e2m1x8_to_f16x2x4(c, f);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&f[i]));
    o[i] = pack_bf16x2(descale * (s * v.x), descale * (s * v.y));
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

template <bool kInv>
__global__ void __launch_bounds__(256) kv4_write_kernel(Kv4WriteParams p) {
  const long long w = ((long long)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  const int lane = threadIdx.x & 31;
  if (w >= p.T * p.Hkv) return;  // whole warps
  const long long t = w / p.Hkv;
  const int h = (int)(w - t * p.Hkv);
  const uint4 rk = __ldcs(reinterpret_cast<const uint4*>(p.k + t * p.k_stride + (long long)h * kD) + lane);
  const uint4 rv = __ldcs(reinterpret_cast<const uint4*>(p.v + t * p.v_stride + (long long)h * kD) + lane);
  const int slot = __ldg(p.slots + t);
  if (slot < 0 || (long long)slot >= p.num_slots) return;
  const size_t row = (size_t)slot * p.Hkv + h;
  float x[8];
  bf16x8_to_float(rk, x);
  store_row4<kInv>(x, p.k_factor, p.k_pool + row * kCodeBytes, p.scales + row * kScalePair, lane);
  bf16x8_to_float(rv, x);
  store_row4<kInv>(x, p.v_factor, p.v_pool + row * kCodeBytes, p.scales + row * kScalePair + kScaleBytes, lane);
}

__global__ void __launch_bounds__(256) kv4_gather_kernel(Kv4GatherParams p) {
  const long long w = ((long long)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  const int lane = threadIdx.x & 31;
  if (w >= p.N * p.Hkv) return;  // whole warps
  const long long n = w / p.Hkv;
  const int h = (int)(w - n * p.Hkv);
  const int slot = __ldg(p.indices + n);
  uint32_t ck = 0u, cv = 0u, sk = 0u, sv = 0u;  // an index outside the pool reads zeros
  if (slot >= 0 && (long long)slot < p.num_slots) {
    const size_t row = (size_t)slot * p.Hkv + h;
    ck = __ldcs(reinterpret_cast<const uint32_t*>(p.k_pool + row * kCodeBytes) + lane);
    cv = __ldcs(reinterpret_cast<const uint32_t*>(p.v_pool + row * kCodeBytes) + lane);
    sk = __ldcs(p.scales + row * kScalePair + (lane >> 1));
    sv = __ldcs(p.scales + row * kScalePair + kScaleBytes + (lane >> 1));
  }
  const size_t out = (size_t)w * kD;
  reinterpret_cast<uint4*>(p.k_out + out)[lane] = row4_to_bf16(ck, sk, p.k_descale);
  reinterpret_cast<uint4*>(p.v_out + out)[lane] = row4_to_bf16(cv, sv, p.v_descale);
}

}  // namespace

cudaError_t launch_kv4_write(const Kv4WriteParams& p, cudaStream_t stream) {
  const unsigned blocks = (unsigned)((p.T * p.Hkv + 7) / 8);
  if (p.inv) kv4_write_kernel<true><<<blocks, 256, 0, stream>>>(p);
  else kv4_write_kernel<false><<<blocks, 256, 0, stream>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_kv4_gather(const Kv4GatherParams& p, cudaStream_t stream) {
  const unsigned blocks = (unsigned)((p.N * p.Hkv + 7) / 8);
  kv4_gather_kernel<<<blocks, 256, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace gda
