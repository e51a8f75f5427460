// gda_mrope.cu -- the step before attention for the tokens of prompts and of decode
// steps, with rotary positions on several axes (time, height, width of images and
// video): per-head RMSNorm of Q and K, the rotation, and the cache write.
//
// Token t has one position per axis; pair i of the rope_dim / 2 rotated pairs belongs to
// axis a(i) and turns by positions[a(i), t] * inv_freq[i] (rotate-half convention: pair i
// is dimensions i and i + rope_dim / 2).  The projection row of a token is
// [q (Hq*D) | gate (Hq*D) | k (Hkv*D) | v (Hkv*D)].
//
// The angle.  pos * inv_freq in FP32 is off by up to pos * 2^-24 turns' worth of radians
// (0.06 at position 10^6), and FP64 runs at a few operations per clock and SM here.  So
// each frequency is held as a 64-bit fraction of a turn, F = frac(inv_freq / 2 pi) 2^64,
// taken once per block: (pos * F) mod 2^64 is the position on the circle with every whole
// turn dropped by the integer wrap, its upper 32 bits go to sincospi, and the error stays
// below 2^-25 turns at any 32-bit position.
//
// Layout.  A block of 8 warps walks the tokens; per token the first rope_dim / 2 threads
// put cos and sin into shared memory, once for all heads, and each warp takes rows in turn
// (lane l owns dimensions 8l .. 8l + 7: one 16-byte load and store; the rotation partner
// is lane l +- rope_dim / 16).  The loads of a warp's first rows go out before the cos and
// sin are computed.  FP32 arithmetic, one rounding to BF16; a 4-bit cache quantises that
// BF16 value, so its rows equal k_out quantised.  Bound by HBM: every row in once and out
// once.
#include "gda_kernels.h"
#include "gda_kv4.cuh"

namespace gda {

namespace {

constexpr int kMropeWarps = 8;

__device__ __forceinline__ void bf16x8_to_float(const uint4& r, float* f) {
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ uint4 float_to_bf16x8(const float* f) {
  return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                    pack_bf16x2(f[6], f[7]));
}

__global__ void __launch_bounds__(kMropeWarps * 32) mrope_kernel(const __grid_constant__ MropeParams p) {
  __shared__ __align__(16) float s_cos[2][kMropeMaxPairs], s_sin[2][kMropeMaxPairs];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int npair = p.rope_dim / 2;
  const bool trig = (int)threadIdx.x < npair;
  unsigned long long F = 0ull;
  const int* pos = p.positions;
  if (trig) {
    double turns = (double)__ldg(p.inv_freq + threadIdx.x) * 0.15915494309189533577;  // 1 / (2 pi)
    turns -= floor(turns);
    F = (unsigned long long)(turns * 18446744073709551616.0);  // 2^64 (1.0 saturates: one part in 2^64 off)
    pos += (long long)p.pair_axis[threadIdx.x] * p.pos_stride;
  }
  // rows of a token in the order the warps take them: q, k, v (with a cache), gate
  const int n_v = p.pool != 0 ? p.Hkv : 0;
  const int n_g = p.gate_out != nullptr ? p.Hq : 0;
  const int rows = p.Hq + p.Hkv + n_v + n_g;
  auto source = [&](long long t, int r) -> const uint4* {
    const int at = r < p.Hq ? r : r < p.Hq + p.Hkv + n_v ? r + p.Hq : r - p.Hkv - n_v;
    return reinterpret_cast<const uint4*>(p.qgkv + t * p.row_stride + (long long)at * kD) + lane;
  };
  int buf = 0;
  for (long long t = blockIdx.x; t < p.T; t += gridDim.x, buf ^= 1) {
    uint4 next = make_uint4(0u, 0u, 0u, 0u);
    if (warp < rows) next = __ldg(source(t, warp));
    const int slot = p.pool != 0 ? __ldg(p.slots + t) : -1;
    const bool slot_ok = slot >= 0 && (long long)slot < p.num_slots;
    if (trig) {
      const unsigned long long u = (unsigned long long)(long long)__ldg(pos + t) * F;
      float s, c;
      sincospif((float)(int)(u >> 32) * 4.656612873077393e-10f, &s, &c);  // 2^-31: half turns
      s_cos[buf][threadIdx.x] = c;
      s_sin[buf][threadIdx.x] = s;
    }
    __syncthreads();  // (the other buffer's readers of token t - grid passed this barrier before the next write to it)
    for (int r = warp; r < rows; r += kMropeWarps) {
      const uint4 raw = next;
      if (r + kMropeWarps < rows) next = __ldg(source(t, r + kMropeWarps));
      if (r >= p.Hq + p.Hkv) {
        const int h = r - p.Hq - p.Hkv;
        if (h >= n_v) {  // gate: copied out
          reinterpret_cast<uint4*>(p.gate_out + (t * p.Hq + (h - n_v)) * kD)[lane] = raw;
        } else if (slot_ok) {  // v: into its slot
          const size_t row = (size_t)slot * p.Hkv + h;
          if (p.pool == 1) {
            reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.v_pool) + row * kD)[lane] = raw;
          } else {
            float x[8];
            bf16x8_to_float(raw, x);
            store_row4(x, p.v_descale, static_cast<unsigned char*>(p.v_pool) + row * kCodeBytes,
                       p.scales + row * kScalePair + kScaleBytes, lane);
          }
        }
        continue;
      }
      const bool is_q = r < p.Hq;
      float x[8];
      bf16x8_to_float(raw, x);
      const __nv_bfloat16* w = is_q ? p.w_q : p.w_k;
      if (w != nullptr) {
        float ss = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
        const float rinv = 1.0f / sqrtf(ss * (1.0f / kD) + p.eps);
        float wv[8];
        bf16x8_to_float(__ldg(reinterpret_cast<const uint4*>(w) + lane), wv);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = x[i] * rinv * wv[i];
      }
      if (p.rope_dim > 0) {
        const int hl = p.rope_dim / 16;  // lanes holding the first halves of the pairs
        const bool first = lane < hl;
        float y[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = __shfl_sync(0xffffffffu, x[i], (first ? lane + hl : lane - hl) & 31);
        if (lane < 2 * hl) {
          const int pair = 8 * (first ? lane : lane - hl);
          const float sign = first ? -1.0f : 1.0f;
#pragma unroll
          for (int i = 0; i < 8; ++i) x[i] = x[i] * s_cos[buf][pair + i] + sign * (y[i] * s_sin[buf][pair + i]);
        }
      }
      const uint4 o = float_to_bf16x8(x);
      if (is_q) {
        reinterpret_cast<uint4*>(p.q_out + (t * p.Hq + r) * kD)[lane] = o;
      } else {
        const int h = r - p.Hq;
        if (p.k_out != nullptr) reinterpret_cast<uint4*>(p.k_out + (t * p.Hkv + h) * kD)[lane] = o;
        if (slot_ok) {
          const size_t row = (size_t)slot * p.Hkv + h;
          if (p.pool == 1) {
            reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.k_pool) + row * kD)[lane] = o;
          } else {
            bf16x8_to_float(o, x);
            store_row4(x, p.k_descale, static_cast<unsigned char*>(p.k_pool) + row * kCodeBytes,
                       p.scales + row * kScalePair, lane);
          }
        }
      }
    }
  }
}

}  // namespace

cudaError_t launch_mrope(const MropeParams& p, cudaStream_t stream) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  const long long full = 8LL * sms;  // 8 blocks of 256 threads fill an SM
  mrope_kernel<<<(unsigned)(p.T < full ? p.T : full), kMropeWarps * 32, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace gda
