// gda_stage1_fp4.cu -- split-KV decode stage 1 over a 4-bit KV cache, sm_103a.
//
// The pools hold e2m1 codes with an e4m3 scale per 16 head dimensions (gda_kv4.cuh):
//   K = k_descale * e4m3(s) * e2m1(c), V likewise.
// Q stays BF16; the partial O and LSE are those of the other stage-1 kernels, so stage 2
// (FP32 merge, sinks, the gate) is shared.
//
// What bounds it: 288 bytes per (position, KV head) against 1024 of a BF16 cache, so the
// streaming time falls to a quarter while the arithmetic per position stays.  The design
// spends as few instructions per code as it can:
//  * Persistent grid, two CTAs of 6 warps per SM (of 4 warps for pairs of head groups, which
//    hold two sets of accumulators); warp w takes 32-position tiles w, w + W, ... of its CTA's
//    piece.  K and V rows and their scales go through a per-warp ring of two 9 KB stages filled
//    by cp.async a tile ahead (108 KB a CTA in flight or in use; no registers held by loads, 18
//    copy instructions a tile).  A ring row is 128 code bytes followed by its 16 scale bytes: the
//    144-byte pitch that keeps the 16-byte reads below free of bank conflicts is the row itself.
//    Two CTAs keep the pipes busy while one merges or waits: a ragged batch of 224 sequences took
//    125 us with one CTA of 8 warps and three stages, 107 with one of 12 warps, 103 with two of
//    6.  Of 120 us for 8 x 131072 positions (117 now) the copies alone took 109 and the arithmetic
//    alone 100.  No pipe is near its limit (b64_l4096: issue 44 %, ALU 37 %, tensor 20 %): a tile's
//    steps -- scores, maximum, exponentials, transpose, products -- wait for one another in a warp,
//    and 8 to 12 warps an SM are what the registers allow.
//  * A code times its scale is exact in FP16, so cvt.rn.f16x2.e2m1x2 widens a byte (two
//    codes), one packed multiply applies the scale, and the tiles run as m16n8k16 FP16
//    MMAs with FP32 accumulation.  Q goes to FP16 with one power of two per head (its
//    largest magnitude lands in [2^14, 2^15)); that factor and k_descale are folded into
//    the score scale, v_descale into the partial's normalisation.
//  * QK: S^T[32 tok x 8 heads] = K Q^T, two m-tiles.  Lane (g, t) reads dims 64t .. 64t + 63
//    of tokens g, g + 8 (m-tile 0), g + 16, g + 24 (m-tile 1): 32 code bytes and one word of
//    four scales each.  K-step s takes dims 64t + 4s + {0,1} for k-slots (2t, 2t+1) and
//    + {2,3} for (2t+8, 2t+9): byte 2s of the lane's codes and byte 2s + 1, so a byte is
//    one A register; the Q^T fragments use the same order.
//  * PV: O^T[256 x 8] += V^T P^T, two k-steps of 16 tokens.  An A register pairs two
//    tokens of one dimension.  Lane (g, t) reads bytes 16g .. + 15 of its four tokens; two
//    bit-selects on a pair of words turn (codes of T0, codes of T1) into bytes that hold one
//    dimension's code of both tokens -- four registers per two selects -- and the scale
//    pair is (scale of T0, scale of T1).  Row g of m-tile mt is dim 32g + 2mt, row g + 8 the
//    next one.
//  * P is rounded to FP16 for the MMA (it lies in [0, 2^8]: 2^-11 relative, 2^-25 absolute
//    below 2^-14, against the 4-bit V it multiplies).  O is divided by the FP32 sum of the
//    rounded values, so that a head's weights add up to 1; the LSE takes the FP32 sum before
//    the rounding (the second sum: b64_l4096 42.4 -> 42.7 us, 16 heads 51.0 -> 52.4 us).
//  * With more than 8 query heads per KV head, pairs of groups share one read of the rows and
//    one widening of the codes (16 heads, 8 x 32769 positions: 84 -> 58 us; 52 now).
//  * Merge: as in the e4m3 kernel -- each warp leaves its rescaled O^T fragments in ring
//    stage 0, all threads add the slices in a fixed order.  Tile k of a piece lives in stage
//    (k + 1) % 2, so the next piece's first tile is on its way to stage 1 while stage 0 serves
//    the merge.
#include <atomic>

#include "gda_kernels.h"
#include "gda_kv4.cuh"
#include "gda_tc.cuh"

namespace gda {

namespace {

constexpr int kTok4 = 32;         // tokens per warp tile
constexpr int kRow4 = kCodeBytes + kScaleBytes;   // ring row: codes, then scales (144 bytes)
constexpr float kLazyLog2F4 = 8.0f;
static_assert(kRow4 % 32 == 16, "the row pitch keeps 16-byte reads of 8 rows on different banks");

struct Fp4Stage {
  unsigned char k[kTok4][kRow4];
  unsigned char v[kTok4][kRow4];
};
// NG groups of 8 query heads per piece, W warps per CTA
template <int NG, int W>
struct Fp4Smem {
  uint2 qf[NG][16][32];           // Q^T fragments (FP16, scaled), lane order
  Fp4Stage ring[W][2];            // per-warp rings; stage 0 also holds the merge slice
  float mbuf[W][kG];              // each warp's running max
  float lsum[W][kG];              // each warp's rescaled sum of the rounded probabilities
  float esum[W][kG];              // and of those before the rounding (for the LSE)
  unsigned int qmax[NG][kG];      // largest |q| of each head of the piece (float bits)
};
static_assert(sizeof(float4) * 16 * 32 <= sizeof(Fp4Stage), "merge slice fits a ring stage");

__device__ __forceinline__ void mma_f16(float* c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint4 lds_v4(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
  return v;
}
__device__ __forceinline__ uint32_t lds_u16(uint32_t addr) {
  uint32_t v;
  asm volatile("{\n\t.reg .u16 t;\n\tld.shared.u16 t, [%1];\n\tcvt.u32.u16 %0, t;\n\t}" : "=r"(v) : "r"(addr));
  return v;
}
template <bool kAll>
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, uint32_t src_bytes, uint64_t policy) {
  if (kAll)
    asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "l"(policy)
                 : "memory");
  else
    asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2, %3;" ::"r"(dst), "l"(src),
                 "r"(src_bytes), "l"(policy)
                 : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint32_t word4(const uint4& v, int i) {
  return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
}

struct KvRows {  // one KV head's rows of the three pools
  const unsigned char *k, *v, *s;
  uint32_t code_stride, scale_stride;  // bytes between slots
};

// The copies of one tile (tokens of `slot_lane`) as one group: per instruction four rows of
// codes, or 16 rows' scale chunks.  kAll: every slot is a row; else -1 stands for zeros.
template <bool kAll>
__device__ __forceinline__ void issue_tile(Fp4Stage& st, const KvRows& r, int slot_lane, int lane, uint64_t policy) {
  const int sub = lane >> 3, chunk = lane & 7;
  const unsigned char *kc = r.k + 16 * chunk, *vc = r.v + 16 * chunk, *sc = r.s + 16 * (lane & 1);
  const uint32_t dk = smem_u32(&st.k[sub][16 * chunk]), dv = smem_u32(&st.v[sub][16 * chunk]);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int s = __shfl_sync(0xffffffffu, slot_lane, 4 * i + sub);
    const size_t row = kAll ? (size_t)(uint32_t)s : (size_t)max(s, 0);
    cp_async16<kAll>(dk + 4 * i * kRow4, kc + row * r.code_stride, s >= 0 ? 16u : 0u, policy);
    cp_async16<kAll>(dv + 4 * i * kRow4, vc + row * r.code_stride, s >= 0 ? 16u : 0u, policy);
  }
  const uint32_t ds = smem_u32((lane & 1) ? &st.v[lane >> 1][kCodeBytes] : &st.k[lane >> 1][kCodeBytes]);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int s = __shfl_sync(0xffffffffu, slot_lane, 16 * i + (lane >> 1));
    const size_t row = kAll ? (size_t)(uint32_t)s : (size_t)max(s, 0);
    cp_async16<kAll>(ds + 16 * i * kRow4, sc + row * r.scale_stride, s >= 0 ? 16u : 0u, policy);
  }
  cp_commit();
}

template <int NG>
struct Fp4WarpState {
  float o[NG][16][4];
  float m[NG][2], l[NG][2], e[NG][2];  // heads 2t, 2t + 1 of each group: maximum, sum after
                                       // and before the rounding of P
  uint32_t P[NG][4];         // FP16 probabilities, P[.][j] = tokens g + 8j, heads (2t, 2t+1)

  __device__ __forceinline__ void reset() {
#pragma unroll
    for (int n = 0; n < NG; ++n) {
#pragma unroll
      for (int i = 0; i < 16; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) o[n][i][j] = 0.0f;
      m[n][0] = m[n][1] = -INFINITY;
      l[n][0] = l[n][1] = e[n][0] = e[n][1] = 0.0f;
    }
  }

  // S^T of the tile's K rows, then the softmax update; nv tokens of the tile are valid
  __device__ __forceinline__ void qk_softmax(const Fp4Stage& st, const uint2 (*qf)[16][32], int nv, const float (*sl2)[2],
                                             int lane) {
    const int g = lane >> 2, t = lane & 3;
    float acc[NG][4][4];  // [group][m-tile * 2 + k-step parity][4]
#pragma unroll
    for (int n = 0; n < NG; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[n][i][j] = 0.0f;
    const uint32_t row0 = smem_u32(&st.k[g][0]);  // token g + 8j: + 8 j kRow4
    // dims 64t + 32 half .. + 31: two scale blocks
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      uint4 c[4];
      uint32_t sp[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        c[j] = lds_v4(row0 + 8 * j * kRow4 + 32 * t + 16 * half);
        sp[j] = e4m3x2_to_f16x2(lds_u16(row0 + 8 * j * kRow4 + kCodeBytes + 4 * t + 2 * half));
      }
#pragma unroll
      for (int blk = 0; blk < 2; ++blk) {
        uint32_t sc[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) sc[j] = __byte_perm(sp[j], 0u, blk ? 0x3232 : 0x1010);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          uint2 b[NG][2];
#pragma unroll
          for (int n = 0; n < NG; ++n)
#pragma unroll
            for (int k = 0; k < 2; ++k) b[n][k] = qf[n][8 * half + 4 * blk + 2 * i + k][lane];
#pragma unroll
          for (int mt = 0; mt < 2; ++mt) {
            uint32_t f0[4], f1[4];
            e2m1x8_to_f16x2x4(word4(c[2 * mt], 2 * blk + i), f0);
            e2m1x8_to_f16x2x4(word4(c[2 * mt + 1], 2 * blk + i), f1);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const uint32_t a0 = f16x2_mul(f0[2 * k], sc[2 * mt]), a1 = f16x2_mul(f1[2 * k], sc[2 * mt + 1]);
              const uint32_t a2 = f16x2_mul(f0[2 * k + 1], sc[2 * mt]), a3 = f16x2_mul(f1[2 * k + 1], sc[2 * mt + 1]);
#pragma unroll
              for (int n = 0; n < NG; ++n) mma_f16(acc[n][2 * mt + k], a0, a1, a2, a3, b[n][k].x, b[n][k].y);
            }
          }
        }
      }
    }
#pragma unroll
    for (int n = 0; n < NG; ++n) {
      float s[8];  // s[2j], s[2j + 1]: token g + 8j, heads 2t, 2t + 1 (log2 units)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        s[i] = (acc[n][0][i] + acc[n][1][i]) * sl2[n][i & 1];
        s[4 + i] = (acc[n][2][i] + acc[n][3][i]) * sl2[n][i & 1];
      }
      if (nv < kTok4) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (g + 8 * j >= nv) s[2 * j] = s[2 * j + 1] = -INFINITY;
      }
      // Lazy rescale: the reference maxima move only when a score exceeds them by more
      // than kLazyLog2F4, so probabilities stay <= 2^8.  (A NaN score moves no maximum; its
      // probability is NaN, which the sum and the output keep.)
      const float xa0 = fmaxf(fmaxf(s[0], s[2]), fmaxf(s[4], s[6]));
      const float xb0 = fmaxf(fmaxf(s[1], s[3]), fmaxf(s[5], s[7]));
      const bool grow = xa0 > m[n][0] + kLazyLog2F4 || xb0 > m[n][1] + kLazyLog2F4;
      if (__any_sync(0xffffffffu, grow)) {
        float xa = xa0, xb = xb0;
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) {
          xa = fmaxf(xa, __shfl_xor_sync(0xffffffffu, xa, off));
          xb = fmaxf(xb, __shfl_xor_sync(0xffffffffu, xb, off));
        }
        const float na = fmaxf(m[n][0], xa), nb = fmaxf(m[n][1], xb);
        const float aa = safe_exp2_diff(m[n][0], na), ab = safe_exp2_diff(m[n][1], nb);
        l[n][0] *= aa;
        l[n][1] *= ab;
        e[n][0] *= aa;
        e[n][1] *= ab;
        m[n][0] = na;
        m[n][1] = nb;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          o[n][i][0] *= aa;
          o[n][i][1] *= ab;
          o[n][i][2] *= aa;
          o[n][i][3] *= ab;
        }
      }
      // (no score above -inf yet: reference 0, so that -inf gives probability 0)
      const float ra = (m[n][0] == -INFINITY) ? 0.0f : m[n][0], rb = (m[n][1] == -INFINITY) ? 0.0f : m[n][1];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        // (2 ulp, below the normal range 0: FP16's rounding follows, and 2^-126 against a sum of
        // at least 2^-8 does not count)
        const float pa = ex2_approx(s[2 * j] - ra), pb = ex2_approx(s[2 * j + 1] - rb);
        P[n][j] = pack_f16(pa, pb);
        const float2 r = __half22float2(*reinterpret_cast<const __half2*>(&P[n][j]));
        l[n][0] += r.x;
        l[n][1] += r.y;
        e[n][0] += pa;
        e[n][1] += pb;
      }
    }
  }

  // O^T += V^T P^T over the tile's V rows
  __device__ __forceinline__ void pv(const Fp4Stage& st, int lane) {
    const int g = lane >> 2, t = lane & 3;
    uint32_t base = smem_u32(&st.v[2 * t][0]);
#pragma unroll
    for (int ks = 0; ks < 2; ++ks, base += 16 * kRow4) {
      uint32_t b0[NG], b1[NG];
#pragma unroll
      for (int n = 0; n < NG; ++n) {
        b0[n] = movmatrix_trans(ks ? P[n][2] : P[n][0]);
        b1[n] = movmatrix_trans(ks ? P[n][3] : P[n][1]);
      }
      uint4 c[4];       // tokens 16ks + (2t, 2t+1, 2t+8, 2t+9): codes of dims 32g .. + 31
      uint32_t sc[4];   // their scales of blocks 2g, 2g + 1
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t row = base + ((i & 1) + 8 * (i >> 1)) * kRow4;
        c[i] = lds_v4(row + 16 * g);
        sc[i] = lds_u16(row + kCodeBytes + 2 * g);
      }
#pragma unroll
      for (int blk = 0; blk < 2; ++blk) {
        const uint32_t s01 = e4m3x2_to_f16x2(__byte_perm(sc[0], sc[1], blk ? 0x51 : 0x40));
        const uint32_t s23 = e4m3x2_to_f16x2(__byte_perm(sc[2], sc[3], blk ? 0x51 : 0x40));
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int wi = 2 * blk + i;
          const uint32_t x0 = word4(c[0], wi), x1 = word4(c[1], wi), x2 = word4(c[2], wi), x3 = word4(c[3], wi);
          constexpr uint32_t kLow = 0x0F0F0F0Fu;
          uint32_t e01[4], o01[4], e23[4], o23[4];  // even and odd dims: (T0, T1), (T2, T3)
          e2m1x8_to_f16x2x4((x0 & kLow) | ((x1 << 4) & ~kLow), e01);
          e2m1x8_to_f16x2x4(((x0 >> 4) & kLow) | (x1 & ~kLow), o01);
          e2m1x8_to_f16x2x4((x2 & kLow) | ((x3 << 4) & ~kLow), e23);
          e2m1x8_to_f16x2x4(((x2 >> 4) & kLow) | (x3 & ~kLow), o23);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint32_t a0 = f16x2_mul(e01[k], s01), a1 = f16x2_mul(o01[k], s01);
            const uint32_t a2 = f16x2_mul(e23[k], s23), a3 = f16x2_mul(o23[k], s23);
#pragma unroll
            for (int n = 0; n < NG; ++n) mma_f16(o[n][4 * wi + k], a0, a1, a2, a3, b0[n], b1[n]);
          }
        }
      }
    }
  }
};

template <int NG, int W>
__global__ void __launch_bounds__(W * 32, kFp4CtasPerSm) stage1_fp4_kernel(Stage1Params p) {
  extern __shared__ __align__(128) unsigned char smem_raw[];
  Fp4Smem<NG, W>& sm = *reinterpret_cast<Fp4Smem<NG, W>*>(smem_raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x < NG * kG) (&sm.qmax[0][0])[threadIdx.x] = 0u;
  Sched sched;
  sched.begin(p.indptr, p.B, p.Hkv * p.nteam, p.num_splits, gridDim.x, blockIdx.x, p.min_chunk, p.window,
              p.piece_cost, p.rule_kv8);
  const uint64_t policy = l2_policy_evict_first();

  auto nmine_of = [&](int len) -> int {
    const int ntiles = (len + kTok4 - 1) / kTok4;
    return (ntiles > warp) ? (ntiles - warp + W - 1) / W : 0;
  };
  auto tile_n = [&](int k, int len, int nmine) -> int {
    return (k < nmine) ? min(kTok4, len - kTok4 * (warp + W * k)) : 0;
  };
  // slot of token `lane` of this warp's tile k (-1 past the tile's end or for a bad index)
  auto fetch = [&](const int* idx, int k, int len, int nmine) -> int {
    int s = -1;
    if (lane < tile_n(k, len, nmine)) {
      s = __ldg(idx + kTok4 * (warp + W * k) + lane);
      if (p.check_indices && (s < 0 || (long long)s >= p.num_slots)) {
        atomicOr(&p.hdr->error, kErrIndex);
        s = -1;
      }
    }
    return s;
  };
  auto rows_of = [&](const Piece& pp) -> KvRows {
    const size_t h = (size_t)(pp.kvh / p.nteam);
    return {p.k_pool + h * kCodeBytes, p.v_pool + h * kCodeBytes, p.scales + h * kScalePair,
            (uint32_t)p.Hkv * kCodeBytes, (uint32_t)p.Hkv * kScalePair};
  };

  Fp4WarpState<NG> st;
  Fp4Stage* ring = sm.ring[warp];
  int s1 = -1, s2 = -1, s3 = -1;
  auto issue = [&](Fp4Stage& stage, const KvRows& kv, int slot, int n) {
    if (n == kTok4 && !p.check_indices) issue_tile<true>(stage, kv, slot, lane, policy);
    else if (n > 0) issue_tile<false>(stage, kv, slot, lane, policy);
    else cp_commit();  // (an empty group keeps the count)
  };
  // Q^T fragments of a piece: this warp's (group, k-step) items w = warp + r W
  constexpr int kQr = (NG * 16 + W - 1) / W;
  uint2 qraw[kQr];
  auto load_q = [&](const Piece& pp) {
    const int kvh = pp.kvh / p.nteam, pass0 = (pp.kvh - kvh * p.nteam) * NG;
    const __nv_bfloat16* qg = p.q + ((size_t)pp.b * p.Hq + (size_t)kvh * p.G) * kD;
#pragma unroll
    for (int r = 0; r < kQr; ++r) {
      const int w = warp + r * W;
      const int g = lane >> 2, t = lane & 3, hq = kG * (pass0 + (w >> 4)) + g;
      qraw[r] = make_uint2(0u, 0u);  // (heads past the KV head's group are zeros)
      if (w < NG * 16 && hq < p.G)
        qraw[r] = __ldg(reinterpret_cast<const uint2*>(qg + (size_t)hq * kD + 64 * t + 4 * (w & 15)));
    }
  };
  // Head of a piece: the slots of this warp's first four tiles, the copies of its first one
  // and Q (for a pair of groups Q waits: its registers are taken).  For every piece after
  // the first this runs before the previous piece's merge.
  auto piece_head = [&](const Piece& pp) {
    const int* idx = p.indices + pp.base + pp.j0;
    const int len = pp.j1 - pp.j0, nmine = nmine_of(len);
    const int s0 = fetch(idx, 0, len, nmine);
    s1 = fetch(idx, 1, len, nmine);
    s2 = fetch(idx, 2, len, nmine);
    s3 = fetch(idx, 3, len, nmine);
    if (NG == 1) load_q(pp);
    issue(ring[1], rows_of(pp), s0, tile_n(0, len, nmine));
  };

  __syncthreads();  // qmax initialised
  Piece pc;
  bool have = sched.next(pc);
  // an idle CTA exits without the trigger, so stage 2 is placed after it has left
  if (have) pdl_launch_dependents();
  // (a pair of groups loads Q behind its first copies, and so behind those of every CTA: it is
  // sent to the L2 ahead of them, 51.7 -> 51.1 us for 16 heads per KV head, 8 x 32769)
  if (NG > 1 && have && threadIdx.x < NG * kG * 4) {
    const int kvh = pc.kvh / p.nteam, hq = (pc.kvh - kvh * p.nteam) * NG * kG + (int)(threadIdx.x >> 2);
    const __nv_bfloat16* line = p.q + ((size_t)pc.b * p.Hq + (size_t)kvh * p.G + hq) * kD + 64 * (threadIdx.x & 3);
    if (hq < p.G) asm volatile("prefetch.global.L2 [%0];" ::"l"(line));
  }
  if (have) piece_head(pc);
  bool first = true;
  while (have) {
    const KvRows kv = rows_of(pc);
    const int* idx = p.indices + pc.base + pc.j0;
    const int len = pc.j1 - pc.j0;
    const int nmine = nmine_of(len);
    st.reset();
    // tile 1: at once for the first piece; else when the merge is done with stage 0 (below)
    if (first) issue(ring[0], kv, s1, tile_n(1, len, nmine));

    if (NG > 1) load_q(pc);
#pragma unroll
    for (int r = 0; r < kQr; ++r) {
      const int w = warp + r * W;
      if (w >= NG * 16) continue;
      const uint32_t w2[2] = {qraw[r].x, qraw[r].y};
      float mx = 0.0f;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        mx = fmaxf(mx, fabsf(__uint_as_float(w2[j] << 16)));
        mx = fmaxf(mx, fabsf(__uint_as_float(w2[j] & 0xFFFF0000u)));
      }
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      if ((lane & 3) == 0) atomicMax(&sm.qmax[w >> 4][lane >> 2], __float_as_uint(mx));
    }
    __syncthreads();  // also: the previous piece's merge is done with stage 0 and the Q fragments
    if (!first) issue(ring[0], kv, s1, tile_n(1, len, nmine));
    first = false;
    // Q into FP16: one power-of-two factor 2^e per head puts its largest magnitude in
    // [2^14, 2^15) (an infinite or huge q stays its head's affair)
    auto exponent = [&](int n, int head) -> int {
      const unsigned int qm = sm.qmax[n][head];
      const int e = (qm == 0u) ? 0 : 141 - (int)((qm >> 23) & 0xFFu);
      return max(-126, min(127, e));
    };
    float sl2[NG][2];
#pragma unroll
    for (int n = 0; n < NG; ++n)
#pragma unroll
      for (int i = 0; i < 2; ++i) sl2[n][i] = ldexpf(p.scale_log2, -exponent(n, 2 * (lane & 3) + i));
#pragma unroll
    for (int r = 0; r < kQr; ++r) {
      const int w = warp + r * W;
      if (w >= NG * 16) continue;
      const uint32_t x = qraw[r].x, y = qraw[r].y;
      const float f = __uint_as_float((uint32_t)(exponent(w >> 4, lane >> 2) + 127) << 23);
      sm.qf[w >> 4][w & 15][lane] = make_uint2(pack_f16(__uint_as_float(x << 16) * f, __uint_as_float(x & 0xFFFF0000u) * f),
                                               pack_f16(__uint_as_float(y << 16) * f, __uint_as_float(y & 0xFFFF0000u) * f));
    }
    __syncthreads();
    if (threadIdx.x < NG * kG) (&sm.qmax[0][0])[threadIdx.x] = 0u;  // every thread has read it; the next write follows a barrier

    for (int k = 0; k < nmine; ++k) {
      Fp4Stage& cur = ring[(k + 1) & 1];
      cp_wait<1>();
      __syncwarp();
      st.qk_softmax(cur, sm.qf, tile_n(k, len, nmine), sl2, lane);
      st.pv(cur, lane);
      __syncwarp();
      issue(cur, kv, s2, tile_n(k + 2, len, nmine));  // into the stage just read
      s2 = s3;
      s3 = fetch(idx, k + 4, len, nmine);
    }
    cp_wait<0>();
    __syncwarp();

    // look ahead: the next piece's first loads go out before this piece's merge
    Piece nx;
    const bool have_next = sched.next(nx);
    if (have_next) piece_head(nx);

    // ---- merge, group by group: fragment-order slices in stage 0 of the rings, summed in a
    // fixed order
    const int ha = 2 * (lane & 3), hb = ha + 1;
#pragma unroll
    for (int n = 0; n < NG; ++n) {
#pragma unroll
      for (int off = 4; off < 32; off <<= 1) {
        st.l[n][0] += __shfl_xor_sync(0xffffffffu, st.l[n][0], off);
        st.l[n][1] += __shfl_xor_sync(0xffffffffu, st.l[n][1], off);
        st.e[n][0] += __shfl_xor_sync(0xffffffffu, st.e[n][0], off);
        st.e[n][1] += __shfl_xor_sync(0xffffffffu, st.e[n][1], off);
      }
      if (lane < 4) {
        sm.mbuf[warp][ha] = st.m[n][0];
        sm.mbuf[warp][hb] = st.m[n][1];
      }
      __syncthreads();
      {
        float Ma = sm.mbuf[0][ha], Mb = sm.mbuf[0][hb];
#pragma unroll
        for (int x = 1; x < W; ++x) {
          Ma = fmaxf(Ma, sm.mbuf[x][ha]);
          Mb = fmaxf(Mb, sm.mbuf[x][hb]);
        }
        const float fa = (Ma == -INFINITY) ? 0.0f : safe_exp2_diff(st.m[n][0], Ma);
        const float fb = (Mb == -INFINITY) ? 0.0f : safe_exp2_diff(st.m[n][1], Mb);
        float4* slice = reinterpret_cast<float4*>(&ring[0]);
#pragma unroll
        for (int mt = 0; mt < 16; ++mt)
          slice[mt * 32 + lane] =
              make_float4(st.o[n][mt][0] * fa, st.o[n][mt][1] * fb, st.o[n][mt][2] * fa, st.o[n][mt][3] * fb);
        if (lane < 4) {
          sm.lsum[warp][ha] = st.l[n][0] * fa;
          sm.lsum[warp][hb] = st.l[n][1] * fb;
          sm.esum[warp][ha] = st.e[n][0] * fa;
          sm.esum[warp][hb] = st.e[n][1] * fb;
        }
      }
      __syncthreads();
      const long long id = pc.id * NG + n;
      float* op = p.o_part + id * (kG * kD);
      float la = 0.0f, lb = 0.0f;
#pragma unroll
      for (int x = 0; x < W; ++x) {
        la += sm.lsum[x][ha];
        lb += sm.lsum[x][hb];
      }
      const float ia = (la != 0.0f) ? p.v_descale / la : 0.0f;  // a NaN sum makes a NaN partial
      const float ib = (lb != 0.0f) ? p.v_descale / lb : 0.0f;
      for (int mt = warp; mt < 16; mt += W) {
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int x = 0; x < W; ++x) {
          const float4 v = reinterpret_cast<const float4*>(&sm.ring[x][0])[mt * 32 + lane];
          acc.x += v.x;
          acc.y += v.y;
          acc.z += v.z;
          acc.w += v.w;
        }
        const int d0 = 32 * (lane >> 2) + 2 * mt;
        *reinterpret_cast<float2*>(op + ha * kD + d0) = make_float2(acc.x * ia, acc.z * ia);
        *reinterpret_cast<float2*>(op + hb * kD + d0) = make_float2(acc.y * ib, acc.w * ib);
      }
      if (threadIdx.x < kG) {
        float M = sm.mbuf[0][threadIdx.x], lt = 0.0f;
#pragma unroll
        for (int x = 1; x < W; ++x) M = fmaxf(M, sm.mbuf[x][threadIdx.x]);
#pragma unroll
        for (int x = 0; x < W; ++x) lt += sm.esum[x][threadIdx.x];
        // (stage 2 takes the largest LSE as its reference: +inf carries a NaN through it)
        p.lse_part[id * kG + threadIdx.x] = (lt > 0.0f) ? M + log2f(lt) : (lt == 0.0f) ? -INFINITY : INFINITY;
      }
      __syncthreads();  // stage 0, Q fragments and merge buffers free for the next group or piece
    }
    pc = nx;
    have = have_next;
  }
}

template <int NG, int W>
cudaError_t launch_fp4(const Stage1Params& p, int grid, cudaStream_t stream, std::atomic<bool>* attr_set) {
  static_assert(kFp4CtasPerSm * (sizeof(Fp4Smem<NG, W>) + 1024) <= 228 * 1024, "shared memory per SM");
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!attr_set[dev]) {
    e = cudaFuncSetAttribute(stage1_fp4_kernel<NG, W>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)sizeof(Fp4Smem<NG, W>));
    if (e != cudaSuccess) return e;
    attr_set[dev] = true;
  }
  stage1_fp4_kernel<NG, W><<<grid, W * 32, sizeof(Fp4Smem<NG, W>), stream>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_stage1_fp4(const Stage1Params& p, int grid, cudaStream_t stream) {
  static std::atomic<bool> one_set[64], pair_set[64];  // zero-initialised: false
  return p.team == 2 ? launch_fp4<2, 4>(p, grid, stream, pair_set) : launch_fp4<1, 6>(p, grid, stream, one_set);
}

}  // namespace gda
