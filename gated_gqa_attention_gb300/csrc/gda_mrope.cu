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
// taken once per block to the last bit or two: (pos * F) mod 2^64 is the position on the circle
// with every whole turn dropped by the integer wrap.  Its upper 32 bits, off by 2^-31 turns at
// most at any 32-bit position, go to sincospi as FP32 half turns, whose rounding is 2^-25 of a
// half turn at most: the angle is within 2^-23 radians for frequencies below 2^64.
//
// Layout.  A warp takes a token's rows, with no block barrier; when fewer tokens than warps
// are left (a decode step, the end of a prompt) the warps share the tokens' rows evenly (16383
// tokens on 4864 warps: 71 us; with a last pass of a third of the warps 73.6).  Per token a warp
// takes cos and sin of every pair once (lanes stride over the pairs) and reads back those of its
// own dimensions: lane l owns dimensions 8l .. 8l + 7 (one 16-byte load and store a row), the
// partner of a rotated dimension is in lane l +- rope_dim / 16 and comes by a second load of the
// same line (69 us; by four shuffles 70), and the norm weights are folded into cos and sin:
//   y = rinv (x (w cos) +- x_partner (w_partner sin)).
// Two rows are in flight per warp and share the shuffles of their sums of squares.  FP32
// arithmetic, one rounding to BF16; a 4-bit cache quantises that BF16 value, so its rows equal
// k_out quantised.  Bound by HBM for prompts (every row in once and out once: 16383 tokens of 16
// + 2 heads with a BF16 cache at 5.1 TB/s, 62 us with no arithmetic at all; more rows in flight,
// by registers or by prefetches into the L2, make it slower: 82 us), by latency for a decode step.
#include <type_traits>

#include "gda_kernels.h"
#include "gda_kv4.cuh"
#include "gda_tc.cuh"

namespace gda {

namespace {

constexpr int kMropeWarps = 8;   // per block
constexpr int kMropeBlocksPerSm = 4;

// eight BF16 values as four FP32 pairs
__device__ __forceinline__ void unpack(const uint4& r, float2* f) {
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
}
// a BF16 row into row r of a pool of codes
__device__ __forceinline__ void store_bf16_row4(const uint4& v, float factor, int inv, void* pool, unsigned char* scales,
                                                size_t r, int lane) {
  float2 f[4];
  unpack(v, f);
  const float x[8] = {f[0].x, f[0].y, f[1].x, f[1].y, f[2].x, f[2].y, f[3].x, f[3].y};
  unsigned char* codes = static_cast<unsigned char*>(pool) + r * kCodeBytes;
  if (inv) store_row4<true>(x, factor, codes, scales, lane);
  else store_row4<false>(x, factor, codes, scales, lane);
}

// frac(f / 2 pi) * 2^64 modulo 2^64, from f = m 2^-s by a 24 x 128 bit product with
// floor(2^128 / 2 pi): the product is off by less than 2^24, and its bits from 2^(64 + s) on are
// the result, which is therefore off by less than 2 for |f| < 2^64 (s >= -40).  (FP64 arithmetic
// would cost every warp more than the rest of its start.)
__device__ __forceinline__ unsigned long long turn_fraction(float f) {
  const uint32_t b = __float_as_uint(f);
  const int e = (int)((b >> 23) & 0xFFu);
  const unsigned long long m = (b & 0x7FFFFFu) | (e ? 0x800000u : 0u);
  const int s = 150 - (e ? e : 1);
  constexpr unsigned long long kHigh = 0x28BE60DB9391054AULL, kLow = 0x7F09D5F47D4D3770ULL;
  // words of the product: w0 | w1 | w2, from the lowest
  const unsigned long long w0 = m * kLow, t = __umul64hi(m, kLow);
  const unsigned long long w1 = m * kHigh + t, w2 = __umul64hi(m, kHigh) + (w1 < t ? 1ull : 0ull);
  unsigned long long r;
  if (s < 0) r = s > -64 ? (w1 << -s) | (w0 >> (64 + s)) : 0ull;
  else if (s == 0) r = w1;
  else if (s < 64) r = (w1 >> s) | (w2 << (64 - s));
  else r = s < 128 ? w2 >> (s - 64) : 0ull;
  return (b >> 31) ? 0ull - r : r;
}

__global__ void __launch_bounds__(kMropeWarps * 32, kMropeBlocksPerSm) mrope_kernel(const __grid_constant__ MropeParams p, int max_wpt) {
  __shared__ __align__(16) float s_cs[kMropeWarps][2][kMropeMaxPairs];
  __shared__ unsigned long long s_freq[kMropeMaxPairs];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int npair = p.rope_dim / 2, hl = p.rope_dim / 16;  // hl lanes hold the first halves of the pairs
  const bool rot = lane < 2 * hl, first = lane < hl;
  const int partner = rot ? (first ? lane + hl : lane - hl) : lane;
  const int pair0 = 8 * (first ? lane : lane - hl);        // the lane's first pair
  const long long gw = (long long)blockIdx.x * kMropeWarps + warp, nw = (long long)gridDim.x * kMropeWarps;
  const uint4* qgkv = reinterpret_cast<const uint4*>(p.qgkv) + lane;
  const long long pitch = p.row_stride / 8;                // in 16-byte words

  // frequencies as 64-bit fractions of a turn, once per block
  for (int i = threadIdx.x; i < npair; i += kMropeWarps * 32) s_freq[i] = turn_fraction(__ldg(p.inv_freq + i));
  __syncthreads();

  // a token per warp while there are enough, then the rest shared by all warps
  for (long long t0 = 0; t0 < p.T; t0 += nw) {
    const long long left = p.T - t0;
    const int wpt = left >= nw ? 1 : (int)min(nw / left, (long long)max_wpt);
    const int sub = (int)(gw % wpt);
    const long long t = t0 + gw / wpt;
    if (t >= p.T) break;
    const uint4* row = qgkv + t * pitch;
    const int slot = p.pool != 0 ? __ldg(p.slots + t) : -1;
    const bool slot_ok = slot >= 0 && (long long)slot < p.num_slots;
    const size_t cache_row = (size_t)max(slot, 0) * p.Hkv;  // first row of the token's slot
    __syncwarp();  // the previous token's cos and sin have been read
    for (int i = lane; i < npair; i += 32) {
      const int pos = __ldg(p.positions + (long long)p.pair_axis[i] * p.pos_stride + t);
      const unsigned long long u = (unsigned long long)(long long)pos * s_freq[i];
      float s, c;
      sincospif((float)(int)(u >> 32) * 4.656612873077393e-10f, &s, &c);  // 2^-31: half turns
      s_cs[warp][0][i] = c;
      s_cs[warp][1][i] = s;
    }
    __syncwarp();

    // q rows, then k rows: norm and rotation
#pragma unroll 1
    for (int kind = 0; kind < 2; ++kind) {
      const int heads = kind ? p.Hkv : p.Hq;
      int h = kind ? (sub - p.Hq % wpt + wpt) % wpt : sub;  // this warp's first head
      if (h >= heads) continue;
      const uint4* src = row + ((kind ? 2 * p.Hq : 0) + h) * (kD / 8);
      const __nv_bfloat16* w = kind ? p.w_k : p.w_q;
      float2 cw[4], sw[4];  // dims 8 lane + 2i, + 1: the norm weight times cos, the partner's times +-sin
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        cw[i] = make_float2(1.0f, 1.0f);
        sw[i] = make_float2(0.0f, 0.0f);
        if (rot) {
          cw[i] = *reinterpret_cast<const float2*>(&s_cs[warp][0][pair0 + 2 * i]);
          sw[i] = *reinterpret_cast<const float2*>(&s_cs[warp][1][pair0 + 2 * i]);
          if (first) sw[i] = make_float2(-sw[i].x, -sw[i].y);
        }
      }
      if (w != nullptr) {
        float2 a[4], b[4];
        unpack(__ldg(reinterpret_cast<const uint4*>(w) + lane), a);
        unpack(__ldg(reinterpret_cast<const uint4*>(w) + partner), b);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          cw[i] = mul_f32x2(cw[i], a[i]);
          sw[i] = mul_f32x2(sw[i], b[i]);
        }
      }
      uint4* dst = reinterpret_cast<uint4*>(kind ? p.k_out : p.q_out);
      if (dst != nullptr) dst += (t * heads + h) * (kD / 8) + lane;
      const long long pitch_h = (long long)wpt * (kD / 8);  // from one of the warp's heads to the next
      // N rows at once: their loads and sums overlap
      auto rows = [&](auto count) {
        constexpr int N = decltype(count)::value;
        uint4 raw[N], mate[N] = {};
        float rinv[N];
#pragma unroll
        for (int j = 0; j < N; ++j) {
          raw[j] = __ldcs(src + j * pitch_h);
          if (rot) mate[j] = __ldcs(src + j * pitch_h + (partner - lane));
        }
#pragma unroll
        for (int j = 0; j < N; ++j) {
          float2 x[4];
          unpack(raw[j], x);
          float2 ss = mul_f32x2(x[0], x[0]);
#pragma unroll
          for (int i = 1; i < 4; ++i) ss = fma_f32x2(x[i], x[i], ss);
          rinv[j] = ss.x + ss.y;
        }
        auto finish = [&](float sum) -> float { return (w != nullptr) ? rsqrtf(sum * (1.0f / kD) + p.eps) : 1.0f; };
        if constexpr (N == 2) {
          // each half warp sums one of the two rows and they swap results: 6 shuffles, not 10
          const bool up = lane >= 16;
          float sum = up ? rinv[1] : rinv[0];
          sum += __shfl_xor_sync(0xffffffffu, up ? rinv[0] : rinv[1], 16);
#pragma unroll
          for (int off = 8; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
          const float own = finish(sum), other = __shfl_xor_sync(0xffffffffu, own, 16);
          rinv[0] = up ? other : own;
          rinv[1] = up ? own : other;
        } else {
#pragma unroll
          for (int off = 16; off > 0; off >>= 1) rinv[0] += __shfl_xor_sync(0xffffffffu, rinv[0], off);
          rinv[0] = finish(rinv[0]);
        }
#pragma unroll
        for (int j = 0; j < N; ++j) {
          float2 x[4], y[4];
          unpack(raw[j], x);
          const uint4 o = mate[j];
          unpack(o, y);
          uint32_t out[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float2 v = mul_f32x2(x[i], cw[i]);
            if (rot) v = fma_f32x2(y[i], sw[i], v);  // (other lanes' values never reach an unrotated one)
            v = mul_f32x2(v, make_float2(rinv[j], rinv[j]));
            out[i] = bf16x2_rn(v.x, v.y);
          }
          const uint4 o4 = make_uint4(out[0], out[1], out[2], out[3]);
          if (dst != nullptr) dst[j * pitch_h] = o4;
          if (kind && slot_ok) {
            const size_t r = cache_row + h + j * wpt;
            // (later steps read the cache, the next kernel reads q_out and k_out: these stay in the
            // L2 longer; 4864 tokens 19.9 -> 19.3 us)
            if (p.pool == 1) __stcs(reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.k_pool) + r * kD) + lane, o4);
            else store_bf16_row4(o4, p.k_factor, p.inv, p.k_pool, p.scales + r * kScalePair, r, lane);
          }
        }
        h += N * wpt;
        src += N * pitch_h;
        if (dst != nullptr) dst += N * pitch_h;
      };
      while (h + wpt < heads) rows(std::integral_constant<int, 2>());
      while (h < heads) rows(std::integral_constant<int, 1>());
    }
    // v rows into the cache, gate rows out: copies (v quantised for a 4-bit cache)
    if (slot_ok) {
      for (int h = (sub - (p.Hq + p.Hkv) % wpt + wpt) % wpt; h < p.Hkv; h += wpt) {
        const uint4 raw = __ldcs(row + (2LL * p.Hq + p.Hkv + h) * (kD / 8));
        const size_t r = cache_row + h;
        if (p.pool == 1) __stcs(reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.v_pool) + r * kD) + lane, raw);
        else store_bf16_row4(raw, p.v_factor, p.inv, p.v_pool, p.scales + r * kScalePair + kScaleBytes, r, lane);
      }
    }
    if (p.gate_out != nullptr) {
      uint4* dst = reinterpret_cast<uint4*>(p.gate_out + t * p.Hq * kD) + lane;
      const uint4* src = row + (long long)p.Hq * (kD / 8);
#pragma unroll 4
      for (int h = (sub - (p.Hq + 2 * p.Hkv) % wpt + wpt) % wpt; h < p.Hq; h += wpt) dst[h * (kD / 8)] = __ldcs(src + h * (kD / 8));
    }
  }
}

}  // namespace

cudaError_t launch_mrope(const MropeParams& p, cudaStream_t stream) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  // warps per token: as many as there are rows to share while that leaves SMs idle
  const long long warps = (long long)kMropeBlocksPerSm * kMropeWarps * sms;  // resident at once
  const int rows = p.Hq + 2 * p.Hkv + (p.gate_out != nullptr ? p.Hq : 0);
  long long wpt = warps / p.T;
  wpt = wpt < 1 ? 1 : wpt > rows ? rows : wpt;
  long long blocks = (p.T * wpt + kMropeWarps - 1) / kMropeWarps;
  const long long full = warps / kMropeWarps;
  if (blocks > full) blocks = full;
  mrope_kernel<<<(unsigned)blocks, kMropeWarps * 32, 0, stream>>>(p, rows);
  return cudaGetLastError();
}

}  // namespace gda
