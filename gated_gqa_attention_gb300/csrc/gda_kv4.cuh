// gda_kv4.cuh -- the 4-bit KV cache's row format and its device helpers (sm_103a).
//
// A row of K or V (one slot, one KV head, 256 head dimensions) is 128 bytes of e2m1
// codes -- byte i holds dimension 2i in its low half and 2i + 1 in its high half -- and
// 16 e4m3 scales, one per 16 consecutive dimensions:
//   value = descale * e4m3(scale) * e2m1(code),  e2m1 in +-{0, 1/2, 1, 3/2, 2, 3, 4, 6}.
// K codes, V codes and scales are three pools.  The scales of a slot's K row and V row
// lie side by side (16 + 16 bytes = one 32-byte sector), so a row gathered from
// anywhere in the pool costs 128 + 128 + 32 bytes of whole sectors; with a scale pool
// for K and one for V each would fetch a sector to use half of it.
// A code times its scale has at most 6 significant bits and lies in [2^-10, 2688], so
// it is exact in FP16: the tensor-core kernels widen without a rounding.
#pragma once

#include <cuda_fp16.h>

#include "gda_device.cuh"

namespace gda {

constexpr int kBlk4 = 16;                    // head dimensions per scale
constexpr int kCodeBytes = kD / 2;           // codes of one row: 128
constexpr int kScaleBytes = kD / kBlk4;      // scales of one row: 16
constexpr int kScalePair = 2 * kScaleBytes;  // a slot's K scales, then its V scales: 32

// The four code pairs of w as FP16 pairs: f[i] = (low half, high half) of byte i.
__device__ __forceinline__ void e2m1x8_to_f16x2x4(uint32_t w, uint32_t* f) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "mov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(f[0]), "=r"(f[1]), "=r"(f[2]), "=r"(f[3])
      : "r"(w));
}

// Two e4m3 codes (bytes 0 and 1 of w) as an FP16 pair; exact.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t w) {
  uint32_t f;
  asm("{\n\t.reg .b16 l, h;\n\t"
      "mov.b32 {l, h}, %1;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, l;\n\t}"
      : "=r"(f)
      : "r"(w));
  return f;
}

__device__ __forceinline__ uint32_t f16x2_mul(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// The scale code of a block whose largest |value| (already divided by the descale) is
// amax: the nearest e4m3 to amax / 6, at most 448 (so an infinity saturates).
__device__ __forceinline__ uint32_t scale_code(float amax) {
  uint32_t r;
  asm("{\n\t.reg .b16 t;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 t, %1, %2;\n\t"
      "mov.b32 %0, {t, 0};\n\t}"
      : "=r"(r)
      : "f"(0.0f), "f"(__fdiv_rn(amax, 6.0f)));
  return r & 0xFFu;
}

// Eight values (already divided by their block's scale) as e2m1 codes, value i in bits
// 4i: nearest, ties to the even code, beyond 6 to 6.
__device__ __forceinline__ uint32_t e2m1_codes(const float* z) {
  uint32_t r;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(r)
      : "f"(z[0]), "f"(z[1]), "f"(z[2]), "f"(z[3]), "f"(z[4]), "f"(z[5]), "f"(z[6]), "f"(z[7]));
  return r;
}

// One row written by one warp: lane l holds dimensions 8l .. 8l + 7 in x, so two lanes
// share a block.  codes: the row's 128 code bytes; scales: its 16 scale bytes.
//   y = x / descale, s = e4m3(max |y| / 6), code = e2m1(y / s)
// The divisions are IEEE, so the stored bytes follow from the formula alone.  A block
// with a NaN gets the NaN scale (its values then read back as NaN); a block whose scale
// rounds to 0 gets codes 0.
//
// kInv (x are BF16 values and descale is a power of two, `factor` its exact reciprocal; else
// `factor` is the descale): two divisions a block instead of two an element, with the same
// codes.  y = x factor is exact and has 8 significant bits, s has 4, so y / s is either on a
// border between two codes (a value of 3 bits) or at least 2^-8 of it away; y * (1 / s) in
// FP32 is within 2^-22 of y / s, and rounding it to 17 bits puts it on the border exactly
// when y / s is there and leaves it on its side otherwise.
template <bool kInv>
__device__ __forceinline__ void store_row4(const float* x, float factor, unsigned char* codes, unsigned char* scales,
                                           int lane) {
  float y[8], a = 0.0f;
  bool nan = false;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    y[i] = kInv ? x[i] * factor : __fdiv_rn(x[i], factor);
    nan |= y[i] != y[i];
    a = fmaxf(a, fabsf(y[i]));
  }
  a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 1));
  const unsigned bad = __ballot_sync(0xffffffffu, nan);
  uint32_t sc = scale_code(a);
  const float s = __half2float(__ushort_as_half((unsigned short)(e4m3x2_to_f16x2(sc) & 0xFFFFu)));
  uint32_t c = 0u;
  if ((bad >> (lane & 30)) & 3u) {
    sc = 0x7Fu;
  } else if (s > 0.0f) {
    if (kInv) {
      const float r = __fdiv_rn(1.0f, s);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        y[i] = __uint_as_float((__float_as_uint(y[i] * r) + 0x40u) & ~0x7Fu);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = __fdiv_rn(y[i], s);
    }
    c = e2m1_codes(y);
  }
  reinterpret_cast<uint32_t*>(codes)[lane] = c;
  if ((lane & 1) == 0) scales[lane >> 1] = (unsigned char)sc;
}

}  // namespace gda
