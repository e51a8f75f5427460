// gda_prefill_packed.cu -- gated attention over packed prompts (sm_103a): tcgen05 MMAs, TMEM
// operands and accumulators, TMA loads, one persistent CTA per SM.
//
// The sequences lie one after the other in [T, H, 256] tensors (row pitches of their own),
// cu_q / cu_k give their rows.  Per sequence, query i and query head h:
//   keys visible to query i: causal j <= i + (keys - queries), else all of the sequence
//   O   = sum_j softmax_j(scale * q_i . k_j) v_j            (no visible key: O = 0)
//   out = RNE_bf16(RNE_bf16(O) * RNE_bf16(sigmoid(gate)))
//   lse = natural-log log-sum-exp of the visible scaled scores
//
// Work items are (128-query block, query head).  The lengths are on the device, so the blocks
// are found there: all blocks of all sequences ordered by their number n of 128-key tiles,
// descending, then by sequence.  Nothing is sorted -- the number of blocks with at least n
// tiles has a closed form per sequence, so a warp sums it over the batch (lanes stride over
// the sequences) and searches the n that holds a rank, then finds the sequence by a prefix
// sum -- a few hundred cycles for the first item, less for the next ones, ahead of their use.
// CTA c takes the items in snake order (c, 2G - 1 - c, 2G + c, ..), heads fastest: equal shares
// from a descending list, and neighbouring CTAs read the same keys.
//
// What bounds it: the tensor pipe for long prompts (a tile takes 1.47 us, 1.31 at the measured
// BF16 rate; 1.44 with one sum of the probabilities instead of two), and for short ones what an item costs besides its tiles.  With one CTA per item
// that was 11 us (set-up 1.5, first loads 2.7, last PV 1.0, epilogue 3.6, stores 1.5, the next
// CTA's launch 0.7).  Here the next item's K and Q arrive and its first S products run during
// the epilogue, and it is about 5 us (sigmoids and last PV 2.7 to 3, O to shared memory 0.5,
// products and stores 1, the next S 0.3): 6001 tokens of nine prompts x 32 heads (53 to 56 key
// tiles in 11 items per SM) 207 -> 148 us (151 with both
// sums); 12288 tokens x 16 heads with prefixes 472 -> 427 us (436).
// (Measured and dropped: four more warps that run the whole epilogue during the next item's
// tiles, 210 us, or only its sigmoids, 161 us -- both take from the softmax what they save; the
// sigmoids as a loop over registers that move up, or with reciprocals by Newton steps in place
// of the SFU's, 148 to 153 us.)
//
// Shared memory (all of it): the Q tile [128 x 256], K as a ring of three half tiles (128
// keys x 128 dimensions), V as two; at an item's end the V buffers hold its outputs.  TMEM
// (512 columns): two S / P buffers (128 columns each, P written over S as BF16 pairs) and O
// (256 columns).
//  * warp 8: items and TMA loads of Q and K; warp 10: V; warp 9: S = Q K^T (and the TMEM
//    allocation); warp 11: O += P V -- one issuing lane each (a wait in an issuing thread
//    drains the tensor pipe, so S and PV have threads of their own).
//  * warps 0-7: softmax.  Warps w and w + 4 share query rows 32 w .. + 31, 64 of a tile's 128
//    scores each; they agree on the row max through shared memory and keep a running max
//    (moved lazily, by more than 2^8; O is then rescaled in TMEM) and two sums.  P is rounded
//    to BF16 for the MMA (2^-8 relative, as the values it weighs); O is divided by the sum of
//    the rounded probabilities, so that a row's weights add up to 1 and the rounding of its
//    largest one cancels, and lse takes the sum before the rounding.  Before the last tile's PV
//    they zero the V rows past the sequence's end (rows of the next sequence: a NaN there
//    times a probability of 0 would be NaN).
//  * their epilogue: while the last PV runs, the sigmoids of 16 whole rows per warp (the gate
//    rows were sent to the L2 at the item's start); then O / l from TMEM as BF16 into the V
//    buffers (row per lane; the next item's PV may start), and from there times the sigmoid
//    into `out`.
// The rest of the code is kept short (rolled loops, one short wait): the roles run different
// parts of it at a time, and unrolling the outer loops by two made the kernel 1.4 times slower.
// On a timeout the CTA records kErrTimeout, every role stops, waits (bounded) for the copies
// and MMAs it started, the TMEM is freed and the CTA returns.  Warps meet at mbarriers only
// (bounded waits), never at a hardware barrier before the end.
#include <cuda.h>

#include "gda_kernels.h"
#include "gda_prefill.h"
#include "gda_prefill_dev.cuh"

namespace gda {

namespace {

constexpr int kPM = 128;            // query rows per item (MMA M)
constexpr int kPN = 128;            // keys per tile (MMA N of S)
constexpr int kSoftmaxWarps = 8;    // warps 0-7
constexpr int kLoadWarp = 8, kMmaWarp = 9, kLoadWarpV = 10, kPvWarp = 11;
constexpr int kThreads = 12 * 32;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kTmemS = 0, kTmemO = 256;

constexpr uint32_t kBlk = 128 * 128;               // one 64-column block of 128 rows: 16 KiB
constexpr uint32_t kHalf = 2 * kBlk;               // a half tile: 2 column blocks, 32 KiB
constexpr int kKSlots = 3;
constexpr uint32_t kOffQ = 0;                      // Q tile [4 blocks][128 rows][128 B]
constexpr uint32_t kOffK = kOffQ + 4 * kBlk;
constexpr uint32_t kOffV = kOffK + kKSlots * kHalf;
constexpr uint32_t kOffX = kOffV + 2 * kHalf;      // row max exchange [parity][half][row]; an item's
                                                   // sums take the parity its last tile did not
constexpr uint32_t kOffE = kOffX + 2048;           // second halves' sums for lse [row]
constexpr uint32_t kOffBar = kOffE + 512;
constexpr uint32_t kSmemBytes = kOffBar + 512;
static_assert(kSmemBytes <= 227 * 1024, "shared memory per CTA");

struct Seq {
  int q0, nq, k0, nk;  // first query and key row, lengths (clamped to the tensors)
};
struct Item {
  int b, qb;           // sequence (-1: no more items) and its query block
  Seq s;
  int h, ntiles;       // query head; key tiles
};
struct Bars {
  uint64_t qf, q_empty;                             // Q landed; the item's S products have read it
  uint64_t k_full[kKSlots], k_empty[kKSlots], v_full[2], v_empty[2];
  uint64_t s_full[2], p_full[2], p_empty[2];        // per S / P buffer
  uint64_t xm[4][2];                                // per row quarter and tile parity: both maxima stored
  uint64_t pr[4];                                   // per row quarter: both halves' epilogues are here
  uint64_t o_full, o_empty, v_free;                 // the item's O complete; read; its staging read
  uint64_t i_full[2], i_empty[2];                   // item slots
  Item item[2];
  uint32_t tmem;
  int abort;
};
static_assert(sizeof(Bars) <= 512, "barrier block");
constexpr int kItemReaders = 3 + kSoftmaxWarps;  // V loader, both issuers, softmax

// ---- finding the items

__device__ __forceinline__ Seq seq_of(const PrefillParams& p, int b) {
  Seq s;
  const int q0 = __ldg(p.cu_q + b), q1 = __ldg(p.cu_q + b + 1);
  const int k0 = __ldg(p.cu_k + b), k1 = __ldg(p.cu_k + b + 1);
  s.q0 = min(max(q0, 0), p.Sq);
  s.nq = max(min(q1, p.Sq) - s.q0, 0);
  s.k0 = min(max(k0, 0), p.Skv);
  s.nk = max(min(k1, p.Skv) - s.k0, 0);
  return s;
}
// the first query block of s with at least n key tiles, and how many have
__device__ __forceinline__ int first_block(const Seq& s, int n, int causal) {
  if (n <= 0 || !causal) return 0;
  // block j's last visible key min(nk - 1, 128 j + 127 + off) is at least 128 (n - 1)
  const int off = s.nk - s.nq;
  return max(0, n - 1 - ((off + kPN - 1) >> 7));
}
__device__ __forceinline__ int count_blocks(const Seq& s, int n, int causal) {
  const int nb = (s.nq + kPM - 1) >> 7;
  if (n > 0 && s.nk - 1 < kPN * (n - 1)) return 0;
  return max(0, nb - first_block(s, n, causal));
}
// The block of a rank (a whole warp calls it, with ascending ranks): where the last one was
// is kept, so most calls only look at the next sequences.
struct Finder {
  int n = -1, above = 0, upto = 0;  // blocks with more than n key tiles, with at least n
  int b0 = 0, before = 0;           // blocks with exactly n tiles in sequences before b0

  __device__ __forceinline__ Item find(const PrefillParams& p, int rank) {
    const int lane = threadIdx.x & 31;
    Item t = {-1, 0, {0, 0, 0, 0}, 0, 0};
    if (n < 0 || rank >= upto) {  // the n with total(n + 1) <= rank < total(n)
      int lo = 0, hi = n - 1;
      if (n < 0) {
        int top = 0;  // the most keys of any sequence with queries
#pragma unroll 1
        for (int b = lane; b < p.B; b += 32) {
          const Seq s = seq_of(p, b);
          top = max(top, s.nq > 0 ? s.nk : 0);
        }
        hi = (__reduce_max_sync(0xffffffffu, top) + kPN - 1) >> 7;
      }
      n = -1;
#pragma unroll 1
      while (lo <= hi) {
        const int mid = (lo + hi) >> 1;
        int c0 = 0, c1 = 0;
#pragma unroll 1
        for (int b = lane; b < p.B; b += 32) {
          const Seq s = seq_of(p, b);
          c0 += count_blocks(s, mid, p.causal);
          c1 += count_blocks(s, mid + 1, p.causal);
        }
        c0 = __reduce_add_sync(0xffffffffu, c0);
        c1 = __reduce_add_sync(0xffffffffu, c1);
        if (rank >= c0) {
          hi = mid - 1;
        } else if (rank < c1) {
          lo = mid + 1;
        } else {
          n = mid;
          above = c1;
          upto = c0;
          break;
        }
      }
      if (n < 0) return t;  // no such block, nor any after it
      b0 = before = 0;
    }
    // among the blocks with exactly n tiles, in sequence order
    const int r = rank - above;
#pragma unroll 1
    for (; b0 < p.B; b0 += 32) {
      const int b = b0 + lane;
      Seq s = {0, 0, 0, 0};
      if (b < p.B) s = seq_of(p, b);
      const int mine = count_blocks(s, n, p.causal) - count_blocks(s, n + 1, p.causal);
      int incl = mine;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, off);
        if (lane >= off) incl += v;
      }
      const unsigned hit = __ballot_sync(0xffffffffu, before + incl > r);
      if (hit != 0u) {
        const int src = __ffs(hit) - 1;
        t.b = b0 + src;
        t.qb = __shfl_sync(0xffffffffu, first_block(s, n, p.causal) + r - before - (incl - mine), src);
        t.s.q0 = __shfl_sync(0xffffffffu, s.q0, src);
        t.s.nq = __shfl_sync(0xffffffffu, s.nq, src);
        t.s.k0 = __shfl_sync(0xffffffffu, s.k0, src);
        t.s.nk = __shfl_sync(0xffffffffu, s.nk, src);
        t.ntiles = n;
        return t;
      }
      before += __shfl_sync(0xffffffffu, incl, 31);
    }
    return t;
  }
};

}  // namespace

__global__ void __launch_bounds__(kThreads, 1)
    prefill_packed_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                          const __grid_constant__ CUtensorMap tv, const __grid_constant__ PrefillParams p,
                          uint32_t bound) {
  extern __shared__ __align__(1024) unsigned char sm[];
  // the 128-byte swizzled tiles need a 1024-byte aligned base: a misaligned one is reported,
  // not used (the same for every CTA)
  if ((smem_u32(sm) & 1023u) != 0) {
    if (threadIdx.x == 0) atomicOr(p.error, kErrTimeout);
    return;
  }
  Bars& bars = *reinterpret_cast<Bars*>(sm + kOffBar);
  float* xbuf = reinterpret_cast<float*>(sm + kOffX);
  float* ebuf = reinterpret_cast<float*>(sm + kOffE);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    mbar_init(&bars.qf, 1);
    mbar_init(&bars.q_empty, 1);
    for (int x = 0; x < kKSlots; ++x) {
      mbar_init(&bars.k_full[x], 1);
      mbar_init(&bars.k_empty[x], 1);
    }
    for (int x = 0; x < 2; ++x) {
      mbar_init(&bars.v_full[x], 1);
      mbar_init(&bars.v_empty[x], 1);
      mbar_init(&bars.s_full[x], 1);
      mbar_init(&bars.p_full[x], kSoftmaxWarps);
      mbar_init(&bars.p_empty[x], 1);
      mbar_init(&bars.i_full[x], 1);
      mbar_init(&bars.i_empty[x], kItemReaders);
    }
    for (int q4 = 0; q4 < 4; ++q4) {
      mbar_init(&bars.xm[q4][0], 2);
      mbar_init(&bars.xm[q4][1], 2);
      mbar_init(&bars.pr[q4], 2);
    }
    mbar_init(&bars.o_full, 1);
    mbar_init(&bars.o_empty, kSoftmaxWarps);
    mbar_init(&bars.v_free, kSoftmaxWarps);
    bars.abort = 0;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(&bars.tmem, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  // (as a programmatic dependent: the set-up above ran during the previous kernel's end, whose
  // results are visible from here on; the next call's kernel may do the same)
  pdl_wait_prior_grid();
  pdl_launch_dependents();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars.tmem;
  volatile int* abort_flag = &bars.abort;
  auto fail = [&]() {
    if (bars.abort == 0) atomicOr(p.error, kErrTimeout);
    bars.abort = 1;
  };
  // (short: the roles' code shares one instruction cache, and this is in it thirty times.  A
  // limit below the default is the failure-path test's: polls then hardly suspend.)
  const long long limit = p.wait_limit;
  const uint32_t hint = limit < kWaitLimitCycles ? 0u : 10000u;  // ns
  auto wait = [&](uint64_t* bar, int parity) -> bool {
    if (mbar_try_wait_for(bar, parity & 1, hint)) return true;
    const long long t0 = clock64();
#pragma unroll 1
    do {
      if (*abort_flag || clock64() - t0 > limit) return false;
    } while (!mbar_try_wait_for(bar, parity & 1, hint));
    return true;
  };
  // what a role started is waited for with the default limit, whatever the abort flag says
  auto drain = [&](uint64_t* bar, int parity) {
    const long long t0 = clock64();
#pragma unroll 1
    while (!mbar_try_wait(bar, parity & 1) && clock64() - t0 < kWaitLimitCycles) {
    }
  };
  // item i (in slot i % 2) of this CTA, by one lane; its readers release the slot
  auto get_item = [&](int i, Item* t) -> bool {
    if (!wait(&bars.i_full[i & 1], i >> 1)) return false;
    *t = bars.item[i & 1];
    return true;
  };

  // Every role walks the same items.  `it` counts those with key tiles, T the tiles and N
  // = 2 T the half tiles so far: the phases of the barriers follow from them.
  if (warp < kSoftmaxWarps) {
    // ---------------- softmax: warp w owns rows 32 (w % 4) .. + 31 (its TMEM lane quarter) and
    // keys [64 hc, 64 hc + 64) of each tile, hc = w / 4
    const int rg = warp & 3, hc = warp >> 2;
    const int r = 32 * rg + lane;
    const uint32_t t_row = tmem + ((uint32_t)(rg * 32) << 16);
    bool ok = true;
    int it = 0, T = 0;
    for (int i = 0;; ++i) {
      Item t;
      ok = __all_sync(0xffffffffu, get_item(i, &t));
      __syncwarp();
      if (!ok) break;
      if (lane == 0) mbar_arrive(&bars.i_empty[i & 1]);
      if (t.b < 0) break;
      const int i0 = t.qb * kPM, qi = i0 + r, L = t.s.nk, off = t.s.nk - t.s.nq;
      // for the epilogue this warp takes 16 rows: w0 .. of the item, the sequence's first nrow
      const int w0 = 32 * rg + 16 * hc, nrow = min(16, t.s.nq - i0 - w0);
      uint4* ob = reinterpret_cast<uint4*>(p.out + ((size_t)(t.s.q0 + i0 + w0) * p.Hq + t.h) * kD) + lane;
      const __nv_bfloat16* gate_w = p.gate + (long long)(t.s.q0 + i0 + w0) * p.gate_stride + (long long)t.h * kD;
      if (p.fuse_gate && lane < nrow)  // their gate on its way to the L2 while the item is computed
        asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(gate_w + lane * p.gate_stride), "r"(2 * kD) : "memory");
      // running row max (log2 units), the sum of the probabilities as the MMA multiplies them (the
      // weights of a row add up to 1), and their sum before that rounding (for lse)
      float m_run = -INFINITY, l_run = 0.0f, e_run = 0.0f;
#pragma unroll 1
      for (int j = 0; j < t.ntiles; ++j, ++T) {
        const int sb = T & 1, ph = T >> 1;
        ok = __all_sync(0xffffffffu, wait(&bars.s_full[sb], ph));
        if (!ok) break;
        tc_fence_after();
        float s[64];
        tmem_ld32(t_row + kTmemS + sb * kPN + 64 * hc, s);
        tmem_ld32(t_row + kTmemS + sb * kPN + 64 * hc + 32, s + 32);
        tmem_wait_ld();

        const int k0 = j * kPN + 64 * hc;  // key of s[0]
        if ((k0 + 64 > L) || (p.causal && k0 + 63 > i0 + off)) {
          // keys below `n` of the 64 are visible to this row
          const int n = p.causal ? min(L, qi + off + 1) - k0 : L - k0;
#pragma unroll
          for (int c = 0; c < 64; ++c)
            if (c >= n) s[c] = -INFINITY;
        }
        float hm;
        {
          float e4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int c = 0; c < 64; ++c) e4[c & 3] = fmaxf(e4[c & 3], s[c]);
          hm = fmaxf(fmaxf(e4[0], e4[1]), fmaxf(e4[2], e4[3]));
        }
        // the two halves of the row agree on the tile max (parity-buffered slots); after this
        // both have read their S, so P may overwrite it
        xbuf[(sb * 2 + hc) * kPM + r] = hm;
        tc_fence_before();  // this warp's S reads are ordered before the partner's P writes
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars.xm[rg][sb]);
        ok = __all_sync(0xffffffffu, wait(&bars.xm[rg][sb], ph));
        if (!ok) break;
        tc_fence_after();
        const float mx = fmaxf(hm, xbuf[(sb * 2 + (1 - hc)) * kPM + r]) * p.scale_log2;

        // lazy max: it moves only by more than 2^8, so probabilities stay below 2^8 (both
        // halves of a row take the same decisions from the same values)
        float alpha = 1.0f;
        if (mx > m_run + 8.0f) {
          alpha = (m_run == -INFINITY) ? 0.0f : exp2f(m_run - mx);
          l_run *= alpha;
          e_run *= alpha;
          m_run = mx;
        }
        if (j > 0 && __any_sync(0xffffffffu, alpha != 1.0f)) {
          // O must hold PV of the tile before it is rescaled; this warp rescales its half of O
          ok = __all_sync(0xffffffffu, wait(&bars.p_empty[(T - 1) & 1], (T - 1) >> 1));
          if (!ok) break;
          tc_fence_after();
#pragma unroll 1
          for (int c0 = 128 * hc; c0 < 128 * hc + 128; c0 += 32) {
            float o[32];
            tmem_ld32(t_row + kTmemO + c0, o);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] *= alpha;
            tmem_st32(t_row + kTmemO + c0, o);
          }
          tmem_wait_st();
        }
        // p = 2^(s * scale_log2 - m): half a packed FFMA and one SFU op per score (a masked score gives
        // 2^-inf = 0; a row with no visible key yet uses m = 0); P (BF16 pairs) over the first
        // half of the S buffer: keys 64 h .. at columns 32 h ..
        const float mneg = (m_run == -INFINITY) ? 0.0f : -m_run;
        uint32_t w[32];
        float2 l2 = make_float2(0.0f, 0.0f), e2 = l2;
#pragma unroll
        for (int e = 0; e < 32; ++e) {
          const float2 a = fma_f32x2(make_float2(s[2 * e], s[2 * e + 1]), make_float2(p.scale_log2, p.scale_log2),
                                     make_float2(mneg, mneg));
          const float2 x = make_float2(ex2_approx(a.x), ex2_approx(a.y));
          w[e] = bf16x2_rn(x.x, x.y);
          e2 = add_f32x2(e2, x);
          l2 = add_f32x2(l2, make_float2(__uint_as_float(w[e] << 16), __uint_as_float(w[e] & 0xFFFF0000u)));
        }
        l_run += l2.x + l2.y;
        e_run += e2.x + e2.y;
        tmem_st16(t_row + kTmemS + sb * kPN + 32 * hc, w);
        tmem_st16(t_row + kTmemS + sb * kPN + 32 * hc + 16, w + 16);
        tmem_wait_st();
        if ((j + 1) * kPN > L) {
          // the last tile's V rows past the sequence's end become zeros: 256 threads, 16 bytes
          // each, before this tile's PV may start
          // (the previous tile's PV first: until it is done the barriers may be a phase behind, and
          // a wait on the phase after next returns at once)
          ok = __all_sync(0xffffffffu, (T == 0 || wait(&bars.p_empty[(T - 1) & 1], (T - 1) >> 1)) &&
                                           wait(&bars.v_full[0], T) && wait(&bars.v_full[1], T));
          if (!ok) break;
          const int r0 = L - j * kPN;  // rows r0 .. 127 of each 64-dimension block
#pragma unroll 1
          for (int x = tid; x < (kPN - r0) * 32; x += kSoftmaxWarps * 32)
            *reinterpret_cast<uint4*>(sm + kOffV + ((x & 31) >> 3) * kBlk + (r0 + (x >> 5)) * 128 + (x & 7) * 16) =
                make_uint4(0u, 0u, 0u, 0u);
          fence_async_shared();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars.p_full[sb]);
      }
      if (!ok) break;
      // ---- epilogue.  While the last products run: the sigmoids of this warp's 16 rows, lane l
      // dimensions 8l .. 8l + 7 of each (1 without a gate)
      constexpr int kRows = 16;
      uint32_t sg[4 * kRows];
      const long long os = (long long)p.Hq * (kD / 8);
      if (p.fuse_gate) {
        const uint4* gb = reinterpret_cast<const uint4*>(gate_w) + lane;
        const long long gs = p.gate_stride / 8;
#pragma unroll
        for (int y = 0; y < kRows; ++y) {
          const uint4 v = y < nrow ? __ldcs(gb + y * gs) : make_uint4(0u, 0u, 0u, 0u);
          sg[4 * y] = v.x, sg[4 * y + 1] = v.y, sg[4 * y + 2] = v.z, sg[4 * y + 3] = v.w;
        }
#pragma unroll
        for (int y = 0; y < kRows; y += 4) sigmoids<4>(sg + 4 * y, p.table);
      } else {
#pragma unroll
        for (int e = 0; e < 4 * kRows; ++e) sg[e] = 0x3F803F80u;
      }
      unsigned char* stage = sm + kOffV;
      if (t.ntiles > 0) {
        // the row's sum is its two halves' sums: exchanged in the slots of the parity that the
        // last tile did not use (both halves read them before that tile's exchange)
        xbuf[((T & 1) * 2 + hc) * kPM + r] = l_run;
        if (hc == 1) ebuf[r] = e_run;  // (the first half writes lse)
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars.pr[rg]);
        ok = __all_sync(0xffffffffu, wait(&bars.pr[rg], 2 * it));
        if (!ok) break;
        const float l = xbuf[(T & 1) * 2 * kPM + r] + xbuf[((T & 1) * 2 + 1) * kPM + r];
        if (p.lse && hc == 0 && qi < t.s.nq) {
          const float e = e_run + ebuf[r];
          p.lse[(size_t)t.h * p.Sq + t.s.q0 + qi] = (e == 0.0f) ? -INFINITY : (m_run + log2f(e)) * 0.69314718055994530942f;
        }
        const float inv = (l > 0.0f) ? 1.0f / l : 0.0f;  // (a NaN sum comes with NaN in O)
        // a dead row is 0 also where a value that its block's other rows see was not finite
        const uint32_t keep = (l == 0.0f) ? 0u : 0xFFFFFFFFu;
        ok = __all_sync(0xffffffffu, wait(&bars.o_full, it));
        if (!ok) break;
        tc_fence_after();
        // O / l as BF16 into the V buffers (free: the last PV has completed), this warp's 128
        // columns of its 32 rows: [64-column block][row][128 B], 16-byte chunks swizzled by row
#pragma unroll 1
        for (int c0 = 128 * hc; c0 < 128 * hc + 128; c0 += 64) {
          float o[64];
          tmem_ld32(t_row + kTmemO + c0, o);
          tmem_ld32(t_row + kTmemO + c0 + 32, o + 32);
          tmem_wait_ld();
          unsigned char* dst = stage + (c0 >> 6) * kBlk + r * 128;
#pragma unroll
          for (int u = 0; u < 8; ++u) {
            uint32_t b4[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float2 v = mul_f32x2(make_float2(o[8 * u + 2 * e], o[8 * u + 2 * e + 1]), make_float2(inv, inv));
              b4[e] = bf16x2_rn(v.x, v.y) & keep;
            }
            *reinterpret_cast<uint4*>(dst + 16 * (u ^ (r & 7))) = make_uint4(b4[0], b4[1], b4[2], b4[3]);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&bars.o_empty);  // the next item's PV may start
          mbar_arrive(&bars.pr[rg]);
        }
        ok = __all_sync(0xffffffffu, wait(&bars.pr[rg], 2 * it + 1));  // both halves of these rows are staged
        if (!ok) break;
        ++it;
      } else if (p.lse && hc == 0 && qi < t.s.nq) {
        p.lse[(size_t)t.h * p.Sq + t.s.q0 + qi] = -INFINITY;
      }
      {
#pragma unroll
        for (int y = 0; y < kRows; ++y) {
          const int row = w0 + y;  // (a staged row, also past the sequence's last: not stored then)
          uint4 v = make_uint4(0u, 0u, 0u, 0u);
          if (t.ntiles > 0)
            v = *reinterpret_cast<const uint4*>(stage + (lane >> 3) * kBlk + row * 128 + 16 * ((lane & 7) ^ (row & 7)));
          // (a product of two BF16 values, correctly rounded by one instruction)
          v.x = mul_bf16x2(v.x, sg[4 * y]), v.y = mul_bf16x2(v.y, sg[4 * y + 1]);
          v.z = mul_bf16x2(v.z, sg[4 * y + 2]), v.w = mul_bf16x2(v.w, sg[4 * y + 3]);
          if (y < nrow) ob[y * os] = v;
        }
        // (generic accesses to the V buffers before the next copies into them)
        fence_async_shared();
        __syncwarp();
        if (t.ntiles > 0 && lane == 0) mbar_arrive(&bars.v_free);
      }
    }
    if (!ok) fail();
  } else {
    if (warp == kLoadWarp) {
      // ---------------- items, and the TMA loads of Q and of K's halves: half N of the stream
      // goes into slot N % 3 once the MMAs that read the slot's previous half have completed
      const uint32_t G = gridDim.x, c = blockIdx.x;
      int it = 0, slot = 0, use = 0, armed[kKSlots] = {}, armed_q = 0;  // slot = N % 3, use = N / 3
      Finder finder;
      const int gsz = p.Hq / p.Hkv;  // query heads per KV head
      bool ok = true;
      auto item_at = [&](int i) -> Item {
        Item t = {-1, 0, {0, 0, 0, 0}, 0, 0};
        const uint32_t x = (uint32_t)i * G + ((i & 1) ? G - 1 - c : c);  // (below bound + 2 G < 2^32)
        if (x < bound) {
          const uint32_t rank = x / (uint32_t)p.Hq;
          t = finder.find(p, (int)rank);
          t.h = (int)(x - rank * (uint32_t)p.Hq);
        }
        return t;
      };
      Item t = {-1, 0, {0, 0, 0, 0}, 0, 0}, next = t;
      // (round -1 only finds item 0: one call site of the finder)
#pragma unroll 1
      for (int i = -1;; ++i) {
        t = next;
        if (i >= 0 && lane == 0) {
          if (i >= 2) ok = wait(&bars.i_empty[i & 1], (i >> 1) - 1);
          if (ok) {
            bars.item[i & 1] = t;
            mbar_arrive(&bars.i_full[i & 1]);
          }
        }
        ok = __shfl_sync(0xffffffffu, (int)ok, 0) != 0;
        if (!ok || (i >= 0 && t.b < 0)) break;
        const int halves = 2 * t.ntiles, kvh = t.h / gsz;
        // the K halves [n0, n1) of the item
        auto load_k = [&](int n0, int n1) {
#pragma unroll 1
          for (int n = n0; n < n1 && ok; ++n) {
            if (use > 0) ok = wait(&bars.k_empty[slot], use - 1);
            if (!ok) break;
            ++armed[slot];
            mbar_arrive_expect_tx(&bars.k_full[slot], kHalf);
            // box {64 elements, 128 rows, 2 column blocks}
            tma_load_5d(sm + kOffK + slot * kHalf, &tk, 0, t.s.k0 + (n >> 1) * kPN, 2 * (n & 1), kvh, 0,
                        &bars.k_full[slot]);
            if (++slot == kKSlots) {
              slot = 0;
              ++use;
            }
          }
        };
        if (lane == 0 && halves > 0) {
          // (K's first halves need only free slots, Q the previous item's last S product)
          load_k(0, 2);
          if (ok && it > 0) ok = wait(&bars.q_empty, it - 1);
          if (ok) {
            ++armed_q;
            mbar_arrive_expect_tx(&bars.qf, 4 * kBlk);
            tma_load_5d(sm + kOffQ, &tq, 0, t.s.q0 + t.qb * kPM, 0, t.h, 0, &bars.qf);
          }
          ++it;
        }
        __syncwarp();
        // the next item, and its Q and first K tile on their way to the L2, while this one runs
        next = item_at(i + 1);
        if (lane == 0) {
          if (next.b >= 0 && next.ntiles > 0) {
            const int nh = next.h / gsz;
            tma_prefetch_5d(&tq, 0, next.s.q0 + next.qb * kPM, 0, next.h, 0);
            tma_prefetch_5d(&tk, 0, next.s.k0, 0, nh, 0);
            tma_prefetch_5d(&tk, 0, next.s.k0, 2, nh, 0);
          }
          load_k(2, halves);
        }
        ok = __shfl_sync(0xffffffffu, (int)ok, 0) != 0;
        if (!ok) break;
      }
      if (!ok && lane == 0) {
        fail();
        if (armed_q > 0) drain(&bars.qf, armed_q - 1);
        for (int x = 0; x < kKSlots; ++x)
          if (armed[x] > 0) drain(&bars.k_full[x], armed[x] - 1);
      }
    } else if (lane == 0 && warp == kLoadWarpV) {
      // ---------------- V halves: half h of tile T into slot h once PV(T - 1) has read it
      int it = 0, T = 0, armed[2] = {};
      const int gsz = p.Hq / p.Hkv;
      bool ok = true;
      for (int i = 0;; ++i) {
        Item t;
        ok = get_item(i, &t);
        if (!ok) break;
        mbar_arrive(&bars.i_empty[i & 1]);
        if (t.b < 0) break;
        if (t.ntiles == 0) continue;
        const int kvh = t.h / gsz;
        if (it > 0) ok = wait(&bars.v_free, it - 1);  // the previous item's outputs have left the buffers
        ++it;
#pragma unroll 1
        for (int j = 0; j < t.ntiles && ok; ++j, ++T) {
#pragma unroll 1
          for (int x = 0; x < 2; ++x) {
            if (T > 0 && !wait(&bars.v_empty[x], T - 1)) {
              ok = false;
              break;
            }
            ++armed[x];
            mbar_arrive_expect_tx(&bars.v_full[x], kHalf);
            tma_load_5d(sm + kOffV + x * kHalf, &tv, 0, t.s.k0 + j * kPN, 2 * x, kvh, 0, &bars.v_full[x]);
          }
          if (!ok) break;
        }
        if (!ok) break;
      }
      if (!ok) {
        fail();
        for (int x = 0; x < 2; ++x)
          if (armed[x] > 0) drain(&bars.v_full[x], armed[x] - 1);
      }
    } else if (lane == 0 && warp == kMmaWarp) {
      // ---------------- S issuer: S(T) = Q K(T)^T into S buffer T % 2, which P(T - 2) occupied
      const uint32_t sQ = smem_u32(sm + kOffQ), sK = smem_u32(sm + kOffK);
      const uint32_t idS = idesc_bf16(kPM, kPN, 0);
      int it = 0, T = 0, slot = 0, use = 0;
      int done = -1;  // the tile of the last commit to s_full
      bool ok = true;
      for (int i = 0;; ++i) {
        Item t;
        ok = get_item(i, &t);
        if (!ok) break;
        mbar_arrive(&bars.i_empty[i & 1]);
        if (t.b < 0) break;
        if (t.ntiles == 0) continue;
        ok = wait(&bars.qf, it);
#pragma unroll 1
        for (int j = 0; j < t.ntiles && ok; ++j, ++T) {
          const int sb = T & 1;
          const int x0 = slot, u0 = use;
          const int x1 = slot + 1 == kKSlots ? 0 : slot + 1, u1 = slot + 1 == kKSlots ? use + 1 : use;
          ok = wait(&bars.k_full[x0], u0) && wait(&bars.k_full[x1], u1);
          if (ok && T >= 2) ok = wait(&bars.p_empty[sb], (T >> 1) - 1);
          if (!ok) break;
          tc_fence_after();
#pragma unroll
          for (int hh = 0; hh < 2; ++hh) {
            const uint32_t kb = sK + (hh ? x1 : x0) * kHalf;
#pragma unroll
            for (int k8 = 0; k8 < 8; ++k8) {
              const int kk = 8 * hh + k8;  // k-step: head dimensions 16 kk .. 16 kk + 15
              const uint64_t ad = sdesc_sw128(sQ + (kk >> 2) * kBlk + (kk & 3) * 32, 16, 1024);
              const uint64_t bd = sdesc_sw128(kb + ((kk >> 2) & 1) * kBlk + (kk & 3) * 32, 16, 1024);
              umma_bf16_ss(tmem + kTmemS + sb * kPN, ad, bd, idS, kk > 0 ? 1u : 0u);
            }
            umma_commit(&bars.k_empty[hh ? x1 : x0]);
          }
          umma_commit(&bars.s_full[sb]);
          done = T;
          slot = x1 + 1 == kKSlots ? 0 : x1 + 1;
          use = x1 + 1 == kKSlots ? u1 + 1 : u1;
        }
        if (!ok) break;
        umma_commit(&bars.q_empty);  // (every S product of the item)
        ++it;
      }
      if (!ok) {
        fail();
        // the last commit covers every MMA issued before it
        if (done >= 0) drain(&bars.s_full[done & 1], done >> 1);
      }
    } else if (lane == 0 && warp == kPvWarp) {
      // ---------------- PV issuer: O += P(T) V(T), per 128-dimension half of O
      const uint32_t sV = smem_u32(sm + kOffV);
      const uint32_t idO = idesc_bf16(kPM, 128, 1);
      int it = 0, T = 0, done = -1;
      bool ok = true;
      for (int i = 0;; ++i) {
        Item t;
        ok = get_item(i, &t);
        if (!ok) break;
        mbar_arrive(&bars.i_empty[i & 1]);
        if (t.b < 0) break;
        if (t.ntiles == 0) continue;
        if (it > 0) ok = wait(&bars.o_empty, it - 1);  // the epilogue has read the previous item's O
#pragma unroll 1
        for (int j = 0; j < t.ntiles && ok; ++j, ++T) {
          const int pb = T & 1;
          ok = wait(&bars.p_full[pb], T >> 1) && wait(&bars.v_full[0], T) && wait(&bars.v_full[1], T);
          if (!ok) break;
          tc_fence_after();
#pragma unroll
          for (int hh = 0; hh < 2; ++hh) {
#pragma unroll
            for (int kk = 0; kk < 8; ++kk) {
              // V half hh is MN-major (dims contiguous): LBO = stride between its two 64-dim
              // blocks, SBO = 8 key rows; k-step kk = keys 16 kk .. 16 kk + 15, whose P is in
              // columns 8 kk .. 8 kk + 7 of the S buffer
              const uint64_t bd = sdesc_sw128(sV + hh * kHalf + kk * 16 * 128, kBlk, 1024);
              umma_bf16_ts(tmem + kTmemO + 128 * hh, tmem + kTmemS + pb * kPN + 8 * kk, bd, idO,
                           (j > 0 || kk > 0) ? 1u : 0u);
            }
            umma_commit(&bars.v_empty[hh]);
          }
          umma_commit(&bars.p_empty[pb]);
          done = T;
        }
        if (!ok) break;
        umma_commit(&bars.o_full);
        ++it;
      }
      if (!ok) {
        fail();
        if (done >= 0) drain(&bars.p_empty[done & 1], done >> 1);
      }
    }
  }

  // ---- teardown: every role is done (or gave up and waited for what it started)
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

cudaError_t packed_init() {
  return cudaFuncSetAttribute(prefill_packed_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemBytes);
}

cudaError_t launch_prefill_packed(const PrefillParams& params, const void* q, int64_t q_pitch, const void* k,
                                  int64_t k_pitch, const void* v, int64_t v_pitch, const void* gate,
                                  cudaStream_t stream) {
  PrefillParams p = params;
  p.gate = static_cast<const __nv_bfloat16*>(gate);
  CUtensorMap tq, tk, tv;
  const int Sk = p.Skv > 0 ? p.Skv : 1;  // (no keys: nothing is loaded)
  if (!make_map_kv(&tq, q, 1, p.Sq, p.Hq, kPM, 4, q_pitch) || !make_map_kv(&tk, k, 1, Sk, p.Hkv, kPN, 2, k_pitch) ||
      !make_map_kv(&tv, v, 1, Sk, p.Hkv, kPN, 2, v_pitch))
    return cudaErrorInvalidValue;
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  e = prefill_init(dev, stream);
  if (e == cudaSuccess) e = sigmoid_table(&p.table);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  // the most items there can be (the lengths are on the device; CTAs past the last leave at once)
  const long long bound = packed_blocks(p.Sq, p.B) * p.Hq;
  const unsigned grid = (unsigned)(bound < sms ? bound : sms);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = stream;
  // as a programmatic dependent where every item has a CTA and latency counts (300 tokens 12.6 ->
  // 11.8 us); with more items than CTAs the early CTAs only disturb (12288 tokens then 428 -> 438 us)
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = bound <= sms ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, prefill_packed_kernel, tq, tk, tv, p, (uint32_t)bound);
}

}  // namespace gda
