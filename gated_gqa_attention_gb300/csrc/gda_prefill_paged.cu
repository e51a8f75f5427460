// gda_prefill_paged.cu -- gated attention of each sequence's newest tokens over its rows of a paged
// cache (sm_103a): tcgen05 MMAs, TMEM operands and accumulators, rows gathered by slot.
//
// Sequence b has nq new tokens and L positions, the new ones last; its query i is at position
// p = L - nq + i and sees, of the keys j <= p, the last `window` ones and the first `keep` ones
// (all without a window).  Per query head h, with the cache row of position j at slot indices[j]:
//   O   = sum_j e^(s_j) v_j / (e^(sink_h) + sum_j e^(s_j)),  s_j = scale * q . k_j   (no key: O = 0)
//   out = RNE_bf16(RNE_bf16(O) * RNE_bf16(sigmoid(gate))),  lse = log of the divisor
//
// Rows.  The G query heads of a KV head read the same keys, so an item is 256 rows of (token, head)
// pairs of one KV head, token after token: one token of 8 heads fills 8 rows, 32 tokens all 256.
// Its keys come in tiles of 128 positions; tiles that no row of the item sees are left out.
//
// Pairs.  A cluster of two CTAs computes an item, 128 rows in each, by MMAs of the pair (M = 256):
// every gathered row is read once per 256 rows, a CTA gathers half of it (64 keys of K, half the
// dimensions of V) and its shared memory holds three K tiles and two V tiles that way.  Batches
// whose sequences have few rows go by a CTA to an item: 128 rows, tiles of 64 keys (kFewRows).
//
// Shares.  The lengths are on the device.  The items, by sequence, KV head and block, form one
// stream in which an item costs its tiles and a constant; each pair, or lone CTA, takes an equal
// share of it.  An item that a share's end cuts is computed in parts: each share leaves its part (row
// max, sum, unnormalised O in FP32) in the workspace, at most two, and a second kernel joins them in
// the order of the shares, so a result does not depend on which ends first.  What an item costs is
// taken as linear in its number within the sequence, and as constant from the block on whose window
// and first tokens are full, so that sums over items have a closed form (linear to the last block, the prompts under a
// window took 195 us instead of 167).
//
// Roles of a CTA's 16 warps, tied by mbarriers whose every wait is bounded:
//   0-7    softmax and epilogue (row quarter warp % 4, keys or dimensions half warp / 4)
//   8      planner: the share's items, one ahead
//   9      issuer (in rank 0 alone, one lane of it): PV of tile T, then S of tile T + 2
//   10, 11 relays: what landed in the CTA -> proxy fence -> rank 0's barriers
//   12-13  gather K;  14-15 gather Q and V
// BF16 rows are copied by cp.async whose completion arrives at the ring's barrier; codes are copied
// into a ring of each warp's own and widened from there to FP16, which holds every code exactly.
// P stays in TMEM, over the first half of each warp's own scores, so PV reads no shared memory for
// it (P in shared memory with a K ring of two: 869 instead of 814 us for 2048 tokens at 34816).
//
// Roundings to fewer bits: P to the MMA's type, BF16 or FP16 (2^-8 or 2^-11 of a weight; the
// divisor sums the rounded weights, so a row's weights add up to 1; lse sums them unrounded); for
// codes Q to FP16, scaled by a power of two per row; O to BF16 as the formula has it.  Scores, row
// maxima, sums, O and the parts are FP32.
//
// What bounds it (GPU time, without the host's):
//   full rows (2048 tokens at 34816, 8 heads a group, BF16): 640 to 700 us, as the power cap has it, 1620 to
//     1770 TFLOP/s, tensor pipe 80 % busy.  At best 1.43 us a tile, 1.31 at the measured rate of library
//     products.  A tile's chain is softmax 1.1 us, its MMAs and the hops between the two CTAs, with two tiles
//     under way
//   few rows, BF16 (64 sequences of one token, a window of 4096): 98 us for 540 MB, 5.5 TB/s with
//     both kernels.  An item ends with 4-6 us that read nothing
//   few rows, codes (64 sequences of 4 tokens, e4m3): 91 us, 3.1 TB/s, 1.0-1.2 us a tile of 64 keys.
//     No unit is near its limit (tensor pipe 33 %, issue slots 31 %): a tile's steps wait for one
//     another.  (Of 94 us before the issuing warp was converged: without widening 94, without softmax
//     91, without both and the copies 81; eight gathering warps 100.  Four S products under way: 91;
//     widened from registers: twice the time)
//   one short sequence: 12.5 us, of which a share is found and the first rows come in 7-8 us and the
//     parts are joined in 3-4 us
//   single tokens over codes: 48 sequences at 3000 to 5000 positions 65 us (e4m3) and 67 us (4-bit) where the
//     decode kernels take 51 and 38, which have no chain of roles per tile (BF16: 75 and 76)
//   prompts under a window (two of 4097, window 1024): 163 us.  A pair has 6.8 items with 58 tiles: 84 us of tiles,
//     8 of start and join, 7 % more on the fullest share than on average, and 9 us for each item's end
// A TMA gather of four rows a time (tile::gather4) brought 3.95 us a 64 KiB tile, 2.5 TB/s in all,
// against 1.36 us of the cp.async here.
#include <limits.h>

#include <type_traits>

#include "gda.h"
#include "gda_kernels.h"
#include "gda_kv4.cuh"
#include "gda_prefill.h"
#include "gda_prefill_dev.cuh"
#include "gda_prefill_paged.h"

namespace gda {

namespace {

constexpr int kPM = 128;            // rows of an item per CTA
// An item's rows (the MMAs' M), its tiles' keys (N of S) and how many CTAs compute it
template <bool PAIR>
struct Geo {
  static constexpr int kCtas = PAIR ? 2 : 1;
  static constexpr int kRows = kPM * kCtas;
  static constexpr int kKeys = 64 * kCtas;
};
constexpr int kSoftmaxWarps = 8;    // warps 0-7
constexpr int kPlanWarp = 8, kMmaWarp = 9, kRelayWarp = 10;  // relays: 10 for K, 11 for Q and V
constexpr int kGatherWarp = 12;     // the gatherers: the first half of them for K, the others for Q and V
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kTmemS = 0, kTmemO = 256;
constexpr int kGatherers = 4;       // half of them for K, half for Q and V
constexpr int kThreads = 32 * (kGatherWarp + kGatherers);
// registers of a thread (softmax, planner and issuer, gatherers) share out what the block has at its
// launch, 128 each.  Spills are dear here: shared memory leaves the L1 little room.  (Without shares 48
// single tokens over 4 bits take 75 us instead of 69, over e4m3 72 instead of 70)
constexpr int kRegsSoftmax = 168, kRegsIssue = 56, kRegsGather = 120;
static_assert(kRegsSoftmax >= 128 && kRegsIssue <= 128 && kRegsGather <= 128, "the softmax warps grow, the others shrink");
static_assert(256 * kRegsSoftmax + 128 * kRegsIssue + 32 * kGatherers * kRegsGather <= kThreads * 128, "register shares");
constexpr int kRowsK = 64 / (kGatherers / 2), kRowsQ = kPM / (kGatherers / 2);  // of a tile and of Q per gathering warp
// arrivals that make a CTA's part of a tile complete: every copying thread's, or one of each widening warp
template <int KV>
constexpr int kLandings = KV == GDA_KV_BF16 ? 16 * kGatherers : kGatherers / 2;
constexpr int kPlaces = 16 / kGatherers;  // codes: 16-byte pieces of a step per thread

// What an item costs besides its tiles, in half tiles (7 us of a pair's tiles: its last softmax and PV, the
// epilogue, the next one's first S).  With 4, 10, 14 and 18: mixed batch of 4-bit rows 488, 395, 402, 410 us; 64
// sequences of 4 tokens, e4m3, by pairs 130, 125, 125, 127; single tokens and prompts within 2 %.  Lone
// CTAs' tiles are half as long, their items end sooner: 6, 10, 16: 98, 94, 93 us for those sequences.
constexpr int kItemCost = 10;

// The batch's kernel: a CTA to an item (128 rows, tiles of 64 keys) where a sequence has no more than
// kFewRows rows (tokens times G) on average, else a pair (256 rows, 128 keys).  The pair's MMAs take the
// same time for any number of rows, a lone CTA's are half of a tile's; its items end side by side.
// 48 sequences at 3000 to 5000 positions, 8 heads a group, lone against pair: single tokens BF16 79 and
// 84 us, e4m3 70 and 84, 4-bit 68 and 86; 16 tokens 96 and 101, 93 and 109, 92 and 109; 24 tokens (two
// blocks of 128) 155 and 108, 155 and 113, 156 and 114.  63 tokens beside a chunk of 512 (71 rows on
// average), all at 4096: 131 and 139, e4m3 143 and 147; of 1024 (135) 159 and 160, 174 and 168.  One
// sequence of one token: 2-5 % slower.
// The rule knows the tensors' sizes alone: empty sequences and rows of no sequence count, and a few long
// sequences among many short ones go by lone CTAs.  2048 tokens at 18048 beside 300 empty sequences: 495 us
// instead of 338 (e4m3 576, 376); 2000 at 18000 beside 200 single tokens: 615, by pairs 563 (e4m3 694, 554).
constexpr int kFewRows = 128;

constexpr uint32_t kBlk = 128 * 128;               // one 64-column block of 128 rows: 16 KiB
constexpr uint32_t kHalf = 2 * kBlk;               // a CTA's half of a K or V tile: 32 KiB
constexpr uint32_t kKBlk = kBlk / 2;               // K: a 64-column block of its 64 keys

constexpr int kStages = 3;          // steps of codes that a gathering warp has under way
template <int KV>
struct Layout {
  static constexpr int kKSlots = KV == GDA_KV_BF16 ? 3 : 2;
  static constexpr uint32_t kOffQ = 0;                          // [4 blocks][128 rows][128 B]
  static constexpr uint32_t kOffK = kOffQ + 4 * kBlk;
  static constexpr uint32_t kOffV = kOffK + kKSlots * kHalf;
  static constexpr uint32_t kOffX = kOffV + 2 * kHalf;          // row max exchange [parity][half][row]
  static constexpr uint32_t kOffE = kOffX + 2048;               // second halves' sums for lse [row]
  static constexpr uint32_t kOffBar = kOffE + 512;
  static constexpr uint32_t kOffScale = kOffBar + 512;          // codes: [4 items][row] the row's score factor
  static constexpr uint32_t kOffStage = kOffScale + 2048;       // and [gathering warp][step] codes (and scales, 4 bytes each)
  static constexpr uint32_t kStageCodes = 512 * kPlaces;  // of a step, per warp
  static constexpr uint32_t kStageBytes = kStageCodes + (KV == GDA_KV_E2M1 ? kStageCodes / 4 : 0), kStageWarp = kStages * kStageBytes;
  static constexpr uint32_t kBytes = KV == GDA_KV_BF16 ? kOffScale : kOffStage + kGatherers * kStageWarp;
  static_assert(kBytes <= 227 * 1024, "shared memory per CTA");
};

struct Item {
  int b;               // sequence (-1: no more items)
  int q0, nq;          // its first new token, their number
  int kb, L;           // first entry of `indices`, positions
  int h, i;            // KV head, block of 256 rows
  int ta, tb;          // this share's tiles of the item's
  int f, tl;           // tile t holds positions from 128 t (t < f) or 128 (t - f + tl) on
  int lo, hi;          // positions that any row sees: [lo, hi) and those below p.keep
  int part;            // -1: the whole item, else where its part goes
};
struct Cut {           // a place in the stream: block i of KV head h of sequence b, before its tile t
  int b, h, i, t;
};
struct Bars {
  // *_land: this CTA's part of Q, K, V has landed (kLandings arrivals).  In rank 0, where
  // both CTAs arrive: q_full and k_full (both parts have), pv_full (P written and both parts of V),
  // o_empty (O read).  Commits arrive in both CTAs
  uint64_t q_land, q_full, q_empty;                 // (q_empty: the item's S products have read it)
  uint64_t k_land[3], k_full[3], k_empty[3], v_land[2];
  uint64_t s_full[2], pv_full[2], p_empty[2];       // per S / P buffer (p_empty: its PV product is complete, V's slot free)
  uint64_t xm[4][2];                                // per row quarter and tile parity: both maxima stored
  uint64_t pr[4];                                   // per row quarter: both halves' epilogues are here
  uint64_t o_full, o_empty, v_free;                 // the item's O complete; read; its staging read
  uint64_t i_full[2], i_empty[2];                   // item slots
  Item item[2];
  uint32_t tmem;
  int abort;
};
static_assert(sizeof(Bars) <= 512, "barrier block");

// ---- the stream of items

struct Seq {
  int q0, nq, kb, L;   // (clamped to the tensors)
};
__device__ __forceinline__ Seq seq_of(const PagedParams& p, int b) {
  Seq s;
  const int q0 = __ldg(p.cu_q + b), q1 = __ldg(p.cu_q + b + 1);
  const int k0 = __ldg(p.indptr + b), k1 = __ldg(p.indptr + b + 1);
  s.q0 = min(max(q0, 0), p.Tq);
  s.nq = max(min(q1, p.Tq) - s.q0, 0);
  s.kb = min(max(k0, 0), p.nnz);
  s.L = max(min(k1, p.nnz) - s.kb, 0);
  return s;
}
// (a sequence's rows, tokens times G, fit 31 bits with two blocks to spare: the host checks it)
template <bool PAIR>
__device__ __forceinline__ int blocks_of(const PagedParams& p, const Seq& s) {
  return (s.nq * p.G + Geo<PAIR>::kRows - 1) / Geo<PAIR>::kRows;
}
// block i of a sequence: what its rows see, and its tiles
struct Range {
  int lo, hi, f, tl, n;
};
template <bool PAIR>
__device__ __forceinline__ Range range_of(const PagedParams& p, const Seq& s, int i) {
  constexpr int kRowsI = Geo<PAIR>::kRows, kPN = Geo<PAIR>::kKeys;
  Range r;
  const int ta = (int)((unsigned)(i * kRowsI) / (unsigned)p.G);                              // first and last token
  const int tb = min(s.nq - 1, (int)((unsigned)(i * kRowsI + kRowsI - 1) / (unsigned)p.G));
  const int off = s.L - s.nq;
  r.hi = max(off + tb + 1, 0);
  r.lo = p.window > 0 ? (int)min(max((long long)off + ta - p.window + 1, 0LL), (long long)r.hi) : 0;
  const int th = (int)(((unsigned)r.hi + kPN - 1) / kPN);
  r.tl = r.lo / kPN;
  r.f = min((int)(((unsigned)min(p.keep, r.lo) + kPN - 1) / kPN), r.tl);
  r.n = r.f + th - r.tl;
  return r;
}
// Costs of a sequence's blocks, per KV head: linear up to block `knee`, constant from there.  (Tiles
// grow with the positions up to the last block, or to the first one where the window and the first
// tokens are both full: only from there on does a later row see no more than an earlier one.)
template <bool PAIR>
struct Costs {
  int mt, knee;            // blocks
  long long first, rise;   // the first one's, and 2^16 times what the next one costs more
  __device__ __forceinline__ Costs(const PagedParams& p, const Seq& s) {
    mt = blocks_of<PAIR>(p, s);
    knee = 0;
    first = rise = 0;
    if (mt > 0) {
      const int n0 = range_of<PAIR>(p, s, 0).n;
      first = 2LL * n0 + kItemCost;
      if (mt > 1) {
        knee = mt - 1;
        if (p.window > 0)  // the block of the token whose position is the window's length and p.keep
          knee = (int)min((long long)knee, max(0LL, (long long)p.window + p.keep - s.L + s.nq) * p.G / Geo<PAIR>::kRows + 1);
        rise = ((2LL * (range_of<PAIR>(p, s, knee).n - n0)) << 16) / knee;
      }
    }
  }
  // of the blocks before block i
  __device__ __forceinline__ long long before(int i) const {
    const long long k = min(i, knee);
    return first * i + ((rise * (k * (k - 1) / 2 + (i - k) * knee)) >> 16);
  }
};
// the place at x within a sequence's costs (0 <= x < Hkv * c.before(c.mt))
template <bool PAIR>
__device__ __forceinline__ Cut cut_at(const PagedParams& p, const Seq& s, int b, long long x) {
  const Costs<PAIR> c(p, s);
  const long long per_head = c.before(c.mt);
  Cut r;
  r.b = b;
  r.h = (int)((unsigned long long)x / (unsigned long long)per_head);
  x -= r.h * per_head;
  int lo = 0, hi = c.mt - 1;   // the last block that starts at or before x
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (c.before(mid) <= x) lo = mid;
    else hi = mid - 1;
  }
  r.i = lo;
  const long long at = c.before(lo), cost = c.before(lo + 1) - at;
  r.t = cost > 0 ? (int)((unsigned long long)(range_of<PAIR>(p, s, lo).n * (x - at)) / (unsigned long long)cost) : 0;
  return r;
}
// Where share x of `shares` starts and ends, and how many shares there are.  A whole warp calls it.
struct Share {
  Cut start, end;
  int used;
};
template <bool PAIR>
__device__ __forceinline__ Share share_of(const PagedParams& p, int x, int shares) {
  const int lane = threadIdx.x & 31;
  Seq s = {0, 0, 0, 0};
  long long cost = 0, total = 0;
#pragma unroll 4
  for (int b = lane; b < p.B; b += 32) {
    s = seq_of(p, b);
    const Costs<PAIR> c(p, s);
    cost = p.Hkv * c.before(c.mt);
    total += cost;
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) total += __shfl_xor_sync(0xffffffffu, total, off);
  Share r;
  // none is less than 128 keys' worth
  r.used = (int)max(1LL, min((long long)shares, total * Geo<PAIR>::kKeys / 256));
  // lanes below 16 find the start, the others the end
  const int y = x + (lane >> 4);
  const long long at = y < r.used ? total * y / r.used : total;
  Seq mine = s;
  int mine_b = p.B;
  long long mine_x = 0, sum = 0;
#pragma unroll 1
  for (int b0 = 0; b0 < p.B; b0 += 32) {
    if (p.B > 32) {
      cost = 0;
      if (b0 + lane < p.B) {
        s = seq_of(p, b0 + lane);
        const Costs<PAIR> c(p, s);
        cost = p.Hkv * c.before(c.mt);
      }
    }
    long long upto = cost;  // of the sequences up to the lane's
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const long long v = __shfl_up_sync(0xffffffffu, upto, off);
      if (lane >= off) upto += v;
    }
    upto += sum;
    const long long at0 = __shfl_sync(0xffffffffu, at, 0), at1 = __shfl_sync(0xffffffffu, at, 16);
    // (costs of 0 hold no place: from <= at < upto)
    const unsigned hit0 = __ballot_sync(0xffffffffu, at0 >= upto - cost && at0 < upto);
    const unsigned hit1 = __ballot_sync(0xffffffffu, at1 >= upto - cost && at1 < upto);
    const unsigned hit = lane < 16 ? hit0 : hit1;
    const int src = hit ? __ffs(hit) - 1 : 0;
    Seq t;
    t.q0 = __shfl_sync(0xffffffffu, s.q0, src);
    t.nq = __shfl_sync(0xffffffffu, s.nq, src);
    t.kb = __shfl_sync(0xffffffffu, s.kb, src);
    t.L = __shfl_sync(0xffffffffu, s.L, src);
    const long long from = __shfl_sync(0xffffffffu, upto - cost, src);
    if (hit) {
      mine = t;
      mine_b = b0 + src;
      mine_x = at - from;
    }
    sum = __shfl_sync(0xffffffffu, upto, 31);
    if (sum > at1) break;   // (both are found)
  }
  Cut c = {p.B, 0, 0, 0};
  if (mine_b < p.B) c = cut_at<PAIR>(p, mine, mine_b, mine_x);
  __syncwarp();
  r.start = {__shfl_sync(0xffffffffu, c.b, 0), __shfl_sync(0xffffffffu, c.h, 0), __shfl_sync(0xffffffffu, c.i, 0),
             __shfl_sync(0xffffffffu, c.t, 0)};
  r.end = {__shfl_sync(0xffffffffu, c.b, 16), __shfl_sync(0xffffffffu, c.h, 16), __shfl_sync(0xffffffffu, c.i, 16),
           __shfl_sync(0xffffffffu, c.t, 16)};
  return r;
}

// Eight codes to FP16, a 16-byte chunk.
__device__ __forceinline__ uint4 e4m3x8_to_f16(uint32_t a, uint32_t b) {
  uint4 f;
  asm("{\n\t.reg .b16 a0, a1, b0, b1;\n\t"
      "mov.b32 {a0, a1}, %4;\n\t"
      "mov.b32 {b0, b1}, %5;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a0;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, a1;\n\t"
      "cvt.rn.f16x2.e4m3x2 %2, b0;\n\t"
      "cvt.rn.f16x2.e4m3x2 %3, b1;\n\t}"
      : "=r"(f.x), "=r"(f.y), "=r"(f.z), "=r"(f.w)
      : "r"(a), "r"(b));
  return f;
}
__device__ __forceinline__ uint4 e2m1x8_to_f16(uint32_t w, uint32_t scale2) {
  uint32_t f[4];
  e2m1x8_to_f16x2x4(w, f);
  return make_uint4(f16x2_mul(f[0], scale2), f16x2_mul(f[1], scale2), f16x2_mul(f[2], scale2), f16x2_mul(f[3], scale2));
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }
// one lane of a converged warp, the same one every time
__device__ __forceinline__ bool elect_one() {
  uint32_t e;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
  return e != 0;
}
template <int N>
__device__ __forceinline__ void regs_grow() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void regs_shrink() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }

__device__ __forceinline__ uint32_t f16x2_rn(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}
// a pair of probabilities rounded for the MMA, and the values they stand for
template <int KV>
__device__ __forceinline__ uint32_t round_pair(float2 x) {
  return KV == GDA_KV_BF16 ? bf16x2_rn(x.x, x.y) : f16x2_rn(x.x, x.y);
}
template <int KV>
__device__ __forceinline__ float2 pair_values(uint32_t w) {
  if (KV == GDA_KV_BF16) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}

// kind::f16 instruction descriptor with BF16 or FP16 operands (their type is a bit in each field)
template <int KV>
__host__ __device__ constexpr uint32_t idesc_of(int M, int N, int b_mn) {
  return idesc_bf16(M, N, b_mn) & (KV == GDA_KV_BF16 ? 0xFFFFFFFFu : ~((1u << 7) | (1u << 10)));
}

// log2-domain sink of a row joined to (m, l, e): its weight goes into the sums, m may rise
__device__ __forceinline__ void join_sink(const PagedParams& p, int head, float& m, float& l, float& e, float& w) {
  const float s = __ldg(p.sinks + head) * 1.44269504088896340736f;
  w = 1.0f;  // what O is multiplied by
  if (s > m) {
    w = (m == -INFINITY) ? 0.0f : exp2f(m - s);
    l = l * w + 1.0f;
    e = e * w + 1.0f;
    m = s;
  } else if (s != -INFINITY) {  // (a NaN too)
    const float t = exp2f(s - m);
    l += t;
    e += t;
  }
}
// the lowest n bits (none for n <= 0, all from 64 on)
__device__ __forceinline__ unsigned long long below(int n) { return n <= 0 ? 0ull : ~0ull >> (64 - min(n, 64)); }
__device__ __forceinline__ float lse_of(float m, float e) {
  return (e == 0.0f) ? -INFINITY : (m + log2f(e)) * 0.69314718055994530942f;
}

template <int KV, bool PAIR>
__device__ __forceinline__ void paged_body(const PagedParams& p) {
  using Lay = Layout<KV>;
  constexpr int kCtas = Geo<PAIR>::kCtas, kRowsI = Geo<PAIR>::kRows, kPN = Geo<PAIR>::kKeys, kHK = kPN / 2;
  constexpr int kRowsV = kPN / (kGatherers / 2);   // of a V tile per gathering warp
  constexpr int kKSlots = Lay::kKSlots;
  extern __shared__ __align__(1024) unsigned char sm[];
  // the 128-byte swizzled tiles need a 1024-byte aligned base: a misaligned one is reported,
  // not used (the same for every CTA)
  if ((smem_u32(sm) & 1023u) != 0) {
    pdl_wait_prior_grid();   // (the joining kernel starts when this one is over)
    if (threadIdx.x == 0) {
      atomicOr(p.error, kErrTimeout);
      p.cuts[0] = make_int4(0, 0, 0, 0);
    }
    return;
  }
  Bars& bars = *reinterpret_cast<Bars*>(sm + Lay::kOffBar);
  float* xbuf = reinterpret_cast<float*>(sm + Lay::kOffX);
  float* ebuf = reinterpret_cast<float*>(sm + Lay::kOffE);
  float* qscale = reinterpret_cast<float*>(sm + Lay::kOffScale);
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);   // (so the compiler knows it to be the warp's)
  const int rank = PAIR ? (int)cluster_rank() : 0;
  const int share = (int)blockIdx.x / kCtas, shares = (int)gridDim.x / kCtas;

  if (tid == 0) {
    mbar_init(&bars.q_land, kLandings<KV>);
    mbar_init(&bars.q_full, kCtas);
    mbar_init(&bars.q_empty, 1);
    for (int x = 0; x < kKSlots; ++x) {
      mbar_init(&bars.k_land[x], kLandings<KV>);
      mbar_init(&bars.k_full[x], kCtas);
      mbar_init(&bars.k_empty[x], 1);
    }
    for (int x = 0; x < 2; ++x) {
      mbar_init(&bars.v_land[x], kLandings<KV>);
      mbar_init(&bars.s_full[x], 1);
      mbar_init(&bars.pv_full[x], kCtas * (kSoftmaxWarps + 1));
      mbar_init(&bars.p_empty[x], 1);
      mbar_init(&bars.i_full[x], 1);
      mbar_init(&bars.i_empty[x], 2 + kGatherers + kSoftmaxWarps + (rank == 0 ? 1 : 0));  // relays, gatherers, softmax, issuer
    }
    for (int q4 = 0; q4 < 4; ++q4) {
      mbar_init(&bars.xm[q4][0], 2);
      mbar_init(&bars.xm[q4][1], 2);
      mbar_init(&bars.pr[q4], 2);
    }
    mbar_init(&bars.o_full, 1);
    mbar_init(&bars.o_empty, kCtas * kSoftmaxWarps);
    mbar_init(&bars.v_free, kSoftmaxWarps);
    bars.abort = 0;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    if (PAIR) {
      tmem_alloc_pair(&bars.tmem, kTmemCols);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(&bars.tmem, kTmemCols);
      tmem_relinquish();
    }
  }
  tc_fence_before();
  // (as a programmatic dependent: the set-up above ran during the previous kernel's end, whose
  // results are visible from here on)
  pdl_wait_prior_grid();
  pdl_launch_dependents();

  // all barriers are set up before anything arrives at them (the planner's share is found meanwhile)
  __syncwarp();
  if (PAIR) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  else __syncthreads();
  Share mine = {};
  if (warp == kPlanWarp) mine = share_of<PAIR>(p, share, shares);
  __syncwarp();
  if (PAIR) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, bars.tmem, 0);
  volatile int* abort_flag = &bars.abort;
  auto fail = [&]() {
    if (bars.abort == 0) atomicOr(p.error, kErrTimeout);
    bars.abort = 1;
    if (PAIR)   // (alive until the end)
      asm volatile("st.shared::cluster.u32 [%0], 1;" ::"r"(cluster_addr(&bars.abort, rank ^ 1)) : "memory");
  };
  // (short: the roles' code shares one instruction cache, and this is in it many times.  A
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
  auto arrive_first = [&](uint64_t* bar) {   // rank 0's barrier
    if (PAIR) mbar_arrive_cluster(cluster_addr(bar, 0));
    else mbar_arrive(bar);
  };
  auto commit = [&](uint64_t* bar) {
    if (PAIR) umma_commit_pair(bar);
    else umma_commit(bar);
  };
  // what a role started is waited for with the default limit, whatever the abort flag says
  auto drain = [&](uint64_t* bar, int parity) {
    const long long t0 = clock64();
#pragma unroll 1
    while (!mbar_try_wait(bar, parity & 1) && clock64() - t0 < kWaitLimitCycles) {
    }
  };
  // item i (in slot i % 2) of this CTA; its readers release the slot
  auto get_item = [&](int i, Item* t) -> bool {
    if (!wait(&bars.i_full[i & 1], i >> 1)) return false;
    *t = bars.item[i & 1];
    return true;
  };

  // Every role walks the same items.  `it` counts those with tiles, T the tiles so far, (slot, use) the
  // places of a ring: the phases of the barriers follow from them.
  if (warp < kSoftmaxWarps) {
    regs_grow<kRegsSoftmax>();
    // ---------------- softmax: warp w owns rows 32 (w % 4) .. + 31 (its TMEM lane quarter) and
    // half hc = w / 4 of each tile's keys
    const int rg = warp & 3, hc = warp >> 2;
    const int r = 32 * rg + lane;
    const uint32_t t_row = tmem + ((uint32_t)(rg * 32) << 16);
    bool ok = true;
    int it = 0, T = 0;
    for (int n = 0;; ++n) {
      Item t;
      ok = __all_sync(0xffffffffu, get_item(n, &t));
      __syncwarp();
      if (!ok) break;
      if (lane == 0) mbar_arrive(&bars.i_empty[n & 1]);
      if (t.b < 0) break;
      const int flat0 = t.i * kRowsI + rank * kPM;                          // this CTA's first row
      const int rows = t.nq * p.G - flat0;                                  // (128 at most count)
      const int tok = (int)((unsigned)(flat0 + r) / (unsigned)p.G), head = t.h * p.G + (flat0 + r - tok * p.G);
      // keys that this row sees: below k_hi, and from k_lo on or below p.keep
      const int pos = t.L - t.nq + tok;
      const int k_hi = max(pos + 1, 0), k_lo = p.window > 0 ? (int)max((long long)pos - p.window + 1, 0LL) : 0;
      const bool some = 32 * rg < rows;   // (rows of the warp)
      // for the epilogue this warp takes 16 rows, w0 .. of the item; lane y < 16 knows row y's place
      const int w0 = 32 * rg + 16 * hc, nrow = min(16, rows - w0);
      long long o_at = 0, g_at = 0;       // in 16-byte words
      if (lane < nrow) {
        const int fl = flat0 + w0 + lane;
        const int tk = (int)((unsigned)fl / (unsigned)p.G), hd = t.h * p.G + (fl - tk * p.G);
        o_at = ((long long)(t.q0 + tk) * p.Hq + hd) * (kD / 8);
        g_at = ((t.q0 + tk) * p.gate_stride) / 8 + hd * (kD / 8);
        if (p.gate && t.part < 0)         // the gate on its way to the L2 while the item is computed
          asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(reinterpret_cast<const uint4*>(p.gate) + g_at),
                       "r"(2 * kD) : "memory");
      }
      // running row max (log2 units; for FP16 less a constant), the sum of the probabilities as the MMA multiplies them (the
      // weights of a row add up to 1), and their sum before that rounding (for lse)
      float m_run = -INFINITY, l_run = 0.0f, e_run = 0.0f;
      float factor = p.scale_log2;
#pragma unroll 1
      for (int j = t.ta; j < t.tb; ++j, ++T) {
        const int sb = T & 1, ph = T >> 1;
        ok = __all_sync(0xffffffffu, wait(&bars.s_full[sb], ph));
        if (!ok) break;
        tc_fence_after();
        // (Q's copy was over before the S product began)
        if (KV != GDA_KV_BF16 && j == t.ta && r < rows) factor = qscale[(it & 3) * kPM + r];
        float hm = -INFINITY;
        // (two rolled passes over the scores in TMEM: unrolled over 64 scores in registers, this loop is
        // bound by the fetching of its instructions)
        const uint32_t t_s = t_row + kTmemS + sb * kPN + kHK * hc;      // this warp's scores, then their P
        const int k0 = (j < t.f ? j : j - t.f + t.tl) * kPN + kHK * hc;  // key of the first
        const bool masked = __any_sync(0xffffffffu, k0 + kHK > k_hi || (k0 < k_lo && k0 + kHK > p.keep));
        unsigned long long seen = ~0ull;
        if (masked) seen = below(k_hi - k0) & (~below(k_lo - k0) | below(p.keep - k0));
        if (some) {
#pragma unroll 1
          for (int c0 = 0; c0 < kHK; c0 += 32) {
            float s[32];
            tmem_ld32(t_s + c0, s);
            tmem_wait_ld();
            if (masked) {
              const uint32_t m = (uint32_t)(seen >> c0);
#pragma unroll
              for (int c = 0; c < 32; ++c)
                if (!(m & (1u << c))) s[c] = -INFINITY;
            }
            float e4[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
            for (int c = 4; c < 32; ++c) e4[c & 3] = fmaxf(e4[c & 3], s[c]);
            hm = fmaxf(hm, fmaxf(fmaxf(e4[0], e4[1]), fmaxf(e4[2], e4[3])));
          }
          // (a row past the item's last holds anything: its max stays -inf, so that it decides nothing below)
          if (r >= rows) hm = -INFINITY;
        }
        // the two halves of the row agree on the tile max (parity-buffered slots)
        xbuf[(sb * 2 + hc) * kPM + r] = hm;
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars.xm[rg][sb]);
        ok = __all_sync(0xffffffffu, wait(&bars.xm[rg][sb], ph));
        if (!ok) break;
        if (some) {
          const float mx = fmaxf(hm, xbuf[(sb * 2 + (1 - hc)) * kPM + r]) * factor;
          // lazy max: it moves only by more than 2^8, so probabilities stay below 2^8 (both
          // halves of a row take the same decisions from the same values).  For FP16 it is held
          // 2^7 lower: their range ends at 2^15 instead, and weights down to 2^-21 of the row's
          // largest are normal numbers, those below lose bits under 2^-32 of it.  The difference is compared: beyond 2^24
          // a sum would be rounded, by enough that a probability could reach 2^16, FP16's infinity
          constexpr float kLift = KV == GDA_KV_BF16 ? 0.0f : 7.0f;
          float alpha = 1.0f;
          if (mx - m_run > 8.0f + kLift) {
            alpha = (m_run == -INFINITY) ? 0.0f : exp2f(m_run - (mx - kLift));
            l_run *= alpha;
            e_run *= alpha;
            m_run = mx - kLift;
          }
          if (j > t.ta && __any_sync(0xffffffffu, alpha != 1.0f)) {
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
          // p = 2^(s * factor - m): half a packed FFMA and one SFU op per score (a masked score gives
          // 2^-inf = 0; a row with no visible key yet uses m = 0); P (16-bit pairs) over the first
          // half of this warp's scores
          const float mneg = (m_run == -INFINITY) ? 0.0f : -m_run;
          // huge scores: the product is rounded first, as in the row max, or its rounding error alone
          // could be a large exponent (a row's own choice: its bits do not depend on its neighbours)
          const bool is_huge = fabsf(m_run) > 262144.0f && m_run != -INFINITY;
          const bool huge = __any_sync(0xffffffffu, is_huge);
          float2 l2 = make_float2(0.0f, 0.0f), e2 = l2;
#pragma unroll 1
          for (int c0 = 0; c0 < kHK; c0 += 16) {
            float s[16];
            tmem_ld16(t_s + c0, s);
            tmem_wait_ld();
            if (masked) {
              const uint32_t m = (uint32_t)(seen >> c0);
#pragma unroll
              for (int c = 0; c < 16; ++c)
                if (!(m & (1u << c))) s[c] = -INFINITY;
            }
            float f = factor;
            if (huge) {
              const float before = is_huge ? factor : 1.0f;
#pragma unroll
              for (int c = 0; c < 16; ++c) s[c] *= before;
              if (is_huge) f = 1.0f;
            }
            uint32_t w[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const float2 a = fma_f32x2(make_float2(s[2 * e], s[2 * e + 1]), make_float2(f, f), make_float2(mneg, mneg));
              const float2 x = make_float2(ex2_approx(a.x), ex2_approx(a.y));
              w[e] = round_pair<KV>(x);
              e2 = add_f32x2(e2, x);
              l2 = add_f32x2(l2, pair_values<KV>(w[e]));
            }
            tmem_st8(t_s + c0 / 2, w);
          }
          l_run += l2.x + l2.y;
          e_run += e2.x + e2.y;
          tmem_wait_st();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_first(&bars.pv_full[sb]);
      }
      if (!ok) break;
      const bool tiles = t.tb > t.ta;
      float l = 0.0f, e = 0.0f;
      if (tiles) {
        // the row's sums are its two halves' sums: exchanged in the slots of the parity that the
        // last tile did not use (both halves read them before that tile's exchange)
        xbuf[((T & 1) * 2 + hc) * kPM + r] = l_run;
        if (hc == 1) ebuf[r] = e_run;  // (the first half uses it)
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars.pr[rg]);
        ok = __all_sync(0xffffffffu, wait(&bars.pr[rg], 2 * it));
        if (!ok) break;
        l = xbuf[(T & 1) * 2 * kPM + r] + xbuf[((T & 1) * 2 + 1) * kPM + r];
        if (hc == 0) e = e_run + ebuf[r];
      }
      if (t.part >= 0) {
        // ---- a part of an item: sums and O as they are, for the joining kernel
        const int rr = rank * kPM + r;
        if (hc == 0 && r < rows) p.part_ml[(size_t)t.part * kRowsI + rr] = make_float4(m_run, l, e, 0.0f);
        ok = __all_sync(0xffffffffu, wait(&bars.o_full, it));
        if (!ok) break;
        tc_fence_after();
        if (some) {
          float4* dst = p.part_o + (size_t)t.part * 64 * kRowsI + rr;
#pragma unroll 1
          for (int c0 = 128 * hc; c0 < 128 * hc + 128; c0 += 32) {
            float o[32];
            tmem_ld32(t_row + kTmemO + c0, o);
            tmem_wait_ld();
            if (r < rows) {
#pragma unroll
              for (int u = 0; u < 8; ++u)
                dst[(size_t)((c0 >> 2) + u) * kRowsI] = make_float4(o[4 * u], o[4 * u + 1], o[4 * u + 2], o[4 * u + 3]);
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          arrive_first(&bars.o_empty);
          mbar_arrive(&bars.pr[rg]);
          mbar_arrive(&bars.v_free);
        }
        ok = __all_sync(0xffffffffu, wait(&bars.pr[rg], 2 * it + 1));
        if (!ok) break;
        ++it;
        continue;
      }
      // ---- epilogue of a whole item, four rows at a time (lane l has dimensions 8l .. 8l + 7 of each), the
      // gate of the next four on its way.  Rolled: this code runs once per item, and unrolled its
      // instructions came from the L2 each time (8 rows of a single token: 5 us)
      constexpr int kRows = 4;
      uint32_t sg[4 * kRows];
      auto gate_rows = [&](int y0) {
#pragma unroll
        for (int y = 0; y < kRows; ++y) {
          const long long at = __shfl_sync(0xffffffffu, g_at, (y0 + y) & 31);
          uint4 v = make_uint4(0u, 0u, 0u, 0u);
          if (p.gate && y0 + y < nrow) v = __ldcs(reinterpret_cast<const uint4*>(p.gate) + at + lane);
          sg[4 * y] = v.x, sg[4 * y + 1] = v.y, sg[4 * y + 2] = v.z, sg[4 * y + 3] = v.w;
        }
      };
      gate_rows(0);
      float m = m_run, wo = 1.0f;
      if (p.sinks && r < rows) join_sink(p, head, m, l, e, wo);
      if (p.lse && hc == 0 && r < rows) p.lse[(size_t)head * p.Tq + t.q0 + tok] = lse_of(m, e);
      unsigned char* stage = sm + Lay::kOffV;
      if (tiles) {
        const float inv = (l == 0.0f) ? 0.0f : wo * p.v_digits / l;
        // a dead row is 0 also where a value that its block's other rows see was not finite
        const uint32_t keep = (l == 0.0f || wo == 0.0f) ? 0u : 0xFFFFFFFFu;
        ok = __all_sync(0xffffffffu, wait(&bars.o_full, it));
        if (!ok) break;
        tc_fence_after();
        // O / l as BF16 into the V buffers (free: the last PV has completed), this warp's 128
        // columns of its 32 rows: [64-column block][row][128 B], 16-byte chunks swizzled by row
#pragma unroll 1
        for (int c0 = 128 * hc; c0 < 128 * hc + 128; c0 += 32) {
          float o[32];
          tmem_ld32(t_row + kTmemO + c0, o);
          tmem_wait_ld();
          unsigned char* dst = stage + (c0 >> 6) * kBlk + r * 128;
          const int x7 = ((c0 >> 3) & 7) ^ (r & 7);
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            uint32_t b4[4];
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              float2 v = mul_f32x2(make_float2(o[8 * u + 2 * x], o[8 * u + 2 * x + 1]), make_float2(inv, inv));
              if (KV != GDA_KV_BF16) v = mul_f32x2(v, make_float2(p.v_power, p.v_power));
              b4[x] = bf16x2_rn(v.x, v.y) & keep;
            }
            *reinterpret_cast<uint4*>(dst + 16 * (x7 ^ u)) = make_uint4(b4[0], b4[1], b4[2], b4[3]);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          arrive_first(&bars.o_empty);  // the next item's PV may start
          mbar_arrive(&bars.pr[rg]);
        }
        ok = __all_sync(0xffffffffu, wait(&bars.pr[rg], 2 * it + 1));  // both halves of these rows are staged
        if (!ok) break;
        ++it;
      }
#pragma unroll 1
      for (int y0 = 0; y0 < nrow; y0 += kRows) {
        uint32_t now[4 * kRows];
#pragma unroll
        for (int x = 0; x < 4 * kRows; ++x) now[x] = sg[x];
        gate_rows(y0 + kRows);
        if (p.gate) {
          sigmoids<kRows>(now, p.table);
        } else {
#pragma unroll
          for (int x = 0; x < 4 * kRows; ++x) now[x] = 0x3F803F80u;
        }
#pragma unroll
        for (int y = 0; y < kRows; ++y) {
          const int row = w0 + y0 + y;
          const long long at = __shfl_sync(0xffffffffu, o_at, y0 + y);
          uint4 v = make_uint4(0u, 0u, 0u, 0u);
          if (tiles)
            v = *reinterpret_cast<const uint4*>(stage + (lane >> 3) * kBlk + row * 128 + 16 * ((lane & 7) ^ (row & 7)));
          // (a product of two BF16 values, correctly rounded by one instruction)
          v.x = mul_bf16x2(v.x, now[4 * y]), v.y = mul_bf16x2(v.y, now[4 * y + 1]);
          v.z = mul_bf16x2(v.z, now[4 * y + 2]), v.w = mul_bf16x2(v.w, now[4 * y + 3]);
          if (y0 + y < nrow) reinterpret_cast<uint4*>(p.out)[at + lane] = v;
        }
      }
      // (generic accesses to the V buffers before the next rows go into them)
      fence_async_shared();
      __syncwarp();
      if (tiles && lane == 0) mbar_arrive(&bars.v_free);
    }
    if (!ok) fail();
  } else if (warp < kGatherWarp) {
    regs_shrink<kRegsIssue>();
    if (warp == kPlanWarp) {
      // ---------------- the share's items, one after the other
      if (lane == 0 && rank == 0) {
        if (share == 0) p.cuts[0] = make_int4(mine.used, 0, 0, 0);
        p.cuts[1 + share] = make_int4(mine.start.b, mine.start.h, mine.start.i, mine.start.t);
      }
      const Cut end = mine.end;
      bool ok = true;
      Cut at = mine.start;
      Seq s = {0, 0, 0, 0};
      int mt = 0;
      if (at.b < p.B) {
        s = seq_of(p, at.b);
        mt = blocks_of<PAIR>(p, s);
      }
      if (lane == 0 && rank == 0) p.cuts[1 + shares + share] = make_int4(s.q0, s.nq, 0, 0);
#pragma unroll 1
      for (int n = 0;; ++n) {
        Item t = {};
        t.b = -1;
        const bool last = at.b == end.b && at.h == end.h && at.i == end.i;  // the share ends in this item
        if (at.b < p.B && !(last && end.t <= at.t)) {
          const Range r = range_of<PAIR>(p, s, at.i);
          t.b = at.b;
          t.q0 = s.q0, t.nq = s.nq, t.kb = s.kb, t.L = s.L;
          t.h = at.h, t.i = at.i;
          t.ta = at.t, t.tb = last ? end.t : r.n;
          t.f = r.f, t.tl = r.tl, t.lo = r.lo, t.hi = r.hi;
          t.part = (t.ta > 0) ? 2 * share : (t.tb < r.n) ? 2 * share + 1 : -1;
        }
        if (lane == 0) {
          if (n >= 2) ok = wait(&bars.i_empty[n & 1], (n >> 1) - 1);
          if (ok) {
            bars.item[n & 1] = t;
            mbar_arrive(&bars.i_full[n & 1]);
          }
        }
        ok = __shfl_sync(0xffffffffu, (int)ok, 0) != 0;
        if (!ok || t.b < 0) break;
        if (last) {
          at = end;
          at.b = p.B;
          continue;
        }
        at.t = 0;
        if (++at.i < mt) continue;
        at.i = 0;
        if (++at.h < p.Hkv) continue;
        at.h = 0;
        // the next sequence with new tokens
        ++at.b;
#pragma unroll 1
        for (bool found = false; at.b < p.B && !found;) {
          const int b = at.b + lane;
          int nq = 0;
          if (b < p.B) nq = seq_of(p, b).nq;
          const unsigned any = __ballot_sync(0xffffffffu, nq > 0);
          found = any != 0u;
          at.b += found ? __ffs(any) - 1 : 32;
        }
        at.b = min(at.b, p.B);
        if (at.b < p.B) {
          s = seq_of(p, at.b);
          mt = blocks_of<PAIR>(p, s);
        }
      }
      if (!ok && lane == 0) fail();
    } else if (rank == 0 && warp == kMmaWarp) {
      // ---------------- issuer: S(T) = Q K(T)^T into S buffer T % 2, O += P(T) V(T).  The whole warp goes
      // through the loop and one lane issues, so that the MMAs' operands are in uniform registers (one lane
      // alone in this branch: 2048 tokens 675 us instead of 645).  A wait here lets the tensor pipe run
      // empty, so there are few, all before a group of MMAs: PV(T) and S(T + 2).  One thread's MMAs run in
      // order: S(T + 2) follows PV(T), whose P its scores replace, without a wait between them
      const uint32_t sQ = smem_u32(sm + Lay::kOffQ), sK = smem_u32(sm + Lay::kOffK), sV = smem_u32(sm + Lay::kOffV);
      constexpr uint32_t idS = idesc_of<KV>(kRowsI, kPN, 0), idO = idesc_of<KV>(kRowsI, kD, 1);
      int it = 0, T = 0, slot = 0, use = 0;
      int done_s = -1, done_o = -1;  // tiles of the last commits
      bool ok = true;
      auto mma_ss = [](uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t acc) {
        if (PAIR) umma_pair_ss(d, a, b, id, acc);
        else umma_bf16_ss(d, a, b, id, acc);
      };
      auto mma_ts = [](uint32_t d, uint32_t a, uint64_t b, uint32_t id, uint32_t acc) {
        if (PAIR) umma_pair_ts(d, a, b, id, acc);
        else umma_bf16_ts(d, a, b, id, acc);
      };
      auto issue_s = [&](int x) {
        const uint32_t kb = sK + slot * kHalf;
        if (elect_one()) {
#pragma unroll
          for (int c = 0; c < 4; ++c) {  // 64 head dimensions
            const uint64_t ad = sdesc_sw128(sQ + c * kBlk, 16, 1024), bd = sdesc_sw128(kb + c * kKBlk, 16, 1024);
#pragma unroll
            for (int k = 0; k < 4; ++k)  // 16 each (32 bytes; descriptors count 16)
              mma_ss(tmem + kTmemS + (x & 1) * kPN, ad + 2 * k, bd + 2 * k, idS, (c > 0 || k > 0) ? 1u : 0u);
          }
          commit(&bars.s_full[x & 1]);
          if (KV == GDA_KV_BF16) commit(&bars.k_empty[slot]);
        }
        __syncwarp();
        done_s = x;
        if (++slot == kKSlots) {
          slot = 0;
          ++use;
        }
      };
      auto wait_all = [&](uint64_t* bar, int parity) -> bool { return __all_sync(0xffffffffu, wait(bar, parity)); };
      for (int n = 0;; ++n) {
        ok = wait_all(&bars.i_full[n & 1], n >> 1);
        if (!ok) break;
        const int ib = __shfl_sync(0xffffffffu, bars.item[n & 1].b, 0);
        const int ta = __shfl_sync(0xffffffffu, bars.item[n & 1].ta, 0), tb = __shfl_sync(0xffffffffu, bars.item[n & 1].tb, 0);
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars.i_empty[n & 1]);
        if (ib < 0) break;
        if (tb == ta) continue;
        // (S product x, two tiles ahead of PV product T)
        ok = wait_all(&bars.q_full, it);
        int x = T;
#pragma unroll 1
        for (int j = ta; j < tb + 2 && ok; ++j) {
          const bool more = j < tb;   // S product j of the item, after PV of tile j - 2
          if (more) ok = wait_all(&bars.k_full[slot], use);
          const int pb = T & 1;
          if (j >= ta + 2) {
            if (ok && j == ta + 2 && it > 0) ok = wait_all(&bars.o_empty, it - 1);  // the epilogues have read the previous O
            ok = ok && wait_all(&bars.pv_full[pb], T >> 1);
          }
          if (!ok) break;
          tc_fence_after();
          if (j >= ta + 2) {
            if (elect_one()) {
#pragma unroll
              for (int c = 0; c < 2; ++c) {  // a half's keys; V is MN-major (dims contiguous): LBO = stride between a
                // CTA's 64-dim blocks, SBO = 8 key rows
                const uint64_t bd = sdesc_sw128(sV + pb * kHalf + c * kHK * 128, kPN * 128, 1024);
                const uint32_t a = tmem + kTmemS + pb * kPN + kHK * c;  // (P over the first half of these keys' scores)
#pragma unroll
                for (int k = 0; k < kHK / 16; ++k)  // 16 keys each
                  mma_ts(tmem + kTmemO, a + 8 * k, bd + 128 * k, idO, (j > ta + 2 || c > 0 || k > 0) ? 1u : 0u);
              }
              commit(&bars.p_empty[pb]);
            }
            __syncwarp();
            done_o = T++;
          }
          if (more) {
            issue_s(x++);
            if (j + 1 == tb && elect_one()) commit(&bars.q_empty);   // (every S product of the item)
            __syncwarp();
          }
        }
        if (!ok) break;
        if (elect_one()) commit(&bars.o_full);
        __syncwarp();
        ++it;
      }
      if (!ok) {
        if (lane == 0) fail();
        // the last commits cover every MMA issued before them
        if (done_s >= 0) drain(&bars.s_full[done_s & 1], done_s >> 1);
        if (done_o >= 0) drain(&bars.p_empty[done_o & 1], done_o >> 1);
      }
    } else if (lane == 0 && warp >= kRelayWarp) {
      // ---------------- relays: what has landed in this CTA is passed on to the issuer's barriers (and to
      // the proxy by which the MMAs read it)
      const bool is_v = warp > kRelayWarp;
      const int slots = is_v ? 2 : kKSlots;
      uint64_t* land = is_v ? bars.v_land : bars.k_land;
      uint64_t* full = is_v ? bars.pv_full : bars.k_full;
      int it = 0, slot = 0, use = 0;
      bool ok = true;
      auto pass = [&](uint64_t* from, uint64_t* to, int parity) {
        ok = wait(from, parity);
        if (!ok) return;
        fence_async_shared();
        arrive_first(to);
      };
      for (int n = 0;; ++n) {
        Item t;
        ok = get_item(n, &t);
        if (!ok) break;
        mbar_arrive(&bars.i_empty[n & 1]);
        if (t.b < 0) break;
        if (t.tb == t.ta) continue;
        if (is_v) pass(&bars.q_land, &bars.q_full, it);
#pragma unroll 1
        for (int j = t.ta; j < t.tb && ok; ++j) {
          pass(&land[slot], &full[slot], use);
          if (++slot == slots) {
            slot = 0;
            ++use;
          }
        }
        if (!ok) break;
        ++it;
      }
      if (!ok) fail();
    }
  } else {
    regs_shrink<kRegsGather>();
    // ---------------- gatherers, for K (this CTA's 64 keys of a tile) or for Q and V (128 keys, this CTA's
    // 128 dimensions).  A tile goes into the next slot of its ring once the MMAs that read the slot's
    // previous tile have completed.  BF16 rows are copied asynchronously (cp.async, whose completion
    // arrives at the slot's barrier); codes are copied to a small ring of the warp's and widened from it.
    constexpr int kHalfTeam = kGatherers / 2;
    const int gw = (warp - kGatherWarp) % kHalfTeam;
    const bool is_v = warp >= kGatherWarp + kHalfTeam;
    const int row0 = is_v ? gw * kRowsV : gw * kRowsK;   // this warp's first row of the CTA's part of a tile
    const int key0 = is_v ? row0 : 64 * rank + row0;             // that row's key
    const int slots = is_v ? 2 : kKSlots;
    unsigned char* ring = sm + (is_v ? Lay::kOffV : Lay::kOffK);
    uint64_t* land = is_v ? bars.v_land : bars.k_land;
    uint64_t* empty = is_v ? bars.p_empty : KV == GDA_KV_BF16 ? bars.k_empty : bars.s_full;  // (a ring of two goes by parity, as S does)
    const unsigned char* pool = is_v ? p.v_pool : p.k_pool;
    int it = 0, slot = 0, use = 0;
    bool ok = true;
    // this thread's part of what `bar` counts is on its way, or written
    auto landed = [&](uint64_t* bar) {
      if (KV == GDA_KV_BF16) {
        asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
      } else {
        __syncwarp();       // (one arrival per warp: each thread's would take its turn at the barrier.  A
        if (lane == 0) mbar_arrive(bar);  // fence here would wait for the next tile's loads: the relay has it)
      }
    };
    auto acquire = [&](uint64_t* bar, int parity) -> bool { return __all_sync(0xffffffffu, wait(bar, parity)); };
    for (int n = 0;; ++n) {
      ok = acquire(&bars.i_full[n & 1], n >> 1);
      if (!ok) break;
      const Item t = bars.item[n & 1];
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars.i_empty[n & 1]);
      if (t.b < 0) break;
      if (t.tb == t.ta) continue;
      // four rows per step, eight lanes each: lane l8 of row 4 q + g8 takes 16 bytes of every 128
      const int g8 = lane >> 3, l8 = lane & 7;
      // the slots of this warp's keys of tile j, key0 + lane and (two of them) key0 + 32 + lane: loaded two
      // tiles ahead, looked at when used; kUnseen where no row of the item sees the position
      constexpr int kUnseen = INT_MIN, kPer = kRowsV / 32;
      int n0[kPer], n1[kPer], n2[kPer];
      auto seen_at = [&](int j, int x, int& pos) -> bool {
        pos = (j < t.f ? j : j - t.f + t.tl) * kPN + key0 + lane + 32 * x;
        return (is_v || 32 * x + lane < kRowsK) && j < t.tb && pos < t.hi && (pos >= t.lo || pos < p.keep);
      };
      auto look_up = [&](int j, int* to) {
#pragma unroll
        for (int x = 0; x < kPer; ++x) {
          int pos;
          to[x] = kUnseen;
          if (seen_at(j, x, pos)) to[x] = __ldg(p.indices + t.kb + pos);
        }
      };
      look_up(t.ta, n0);
      look_up(t.ta + 1, n1);
      if (KV != GDA_KV_BF16) look_up(t.ta + 2, n2);
      // the slot of tile j's key x, or -1: zeros.  A row outside the pools reads as zeros and is reported (kUnseen may
      // be what `indices` has for a seen position; to change it there would be to wait for the load)
      auto slot_of = [&](int v, int j, int x) -> int {
        if (v >= 0 && (long long)v < p.num_slots) return v;
        int pos;
        if (v != kUnseen || seen_at(j, x, pos)) atomicOr(p.error, kErrIndex);
        return -1;
      };
      if (is_v && ok) {
        // Q (the previous item's last S product has read it): the item's rows, four rows per
        // step as below; rows past its last stay what they are, and what comes of them goes nowhere
        if (it > 0) ok = acquire(&bars.q_empty, it - 1);
        if (!ok) break;
        const int q0 = gw * kRowsQ, flat0 = t.i * kRowsI + rank * kPM + q0;
        const int rows = min(kRowsQ, t.nq * p.G - flat0);
        const int dt = 4 / p.G, dg = 4 - dt * p.G;     // four rows on
        int tok = (int)((unsigned)(flat0 + g8) / (unsigned)p.G), g = flat0 + g8 - tok * p.G;
        unsigned char* dq = sm + Lay::kOffQ + (q0 + g8) * 128;
#pragma unroll 2
        for (int q = 0; 4 * q < rows; ++q) {
          const bool in = 4 * q + g8 < rows;
          const __nv_bfloat16* src = p.q + (in ? (long long)(t.q0 + tok) * p.q_stride + (long long)(t.h * p.G + g) * kD : 0) + l8 * 8;
          const uint32_t to = smem_u32(dq) + q * 512 + ((l8 ^ ((4 * q + g8) & 7)) << 4);
#pragma unroll
          for (int c = 0; c < 4; ++c) cp_async16(to + c * kBlk, src + 64 * c, in ? 16 : 0);
          tok += dt;
          g += dg;
          if (g >= p.G) {
            g -= p.G;
            ++tok;
          }
        }
        if (KV != GDA_KV_BF16) {
          // to FP16 in place (each thread what it copied), each row times a power of two that brings its
          // largest element to [1, 2): exact but for elements 2^-14 of that and less, which lose bits
          // below 2^-24 of it
          cp_async_wait_all();
#pragma unroll 1
          for (int q = 0; 4 * q < rows; ++q) {
            unsigned char* at = dq + q * 512 + ((l8 ^ ((4 * q + g8) & 7)) << 4);
            uint4 raw[4];
            uint32_t top = 0u;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              raw[c] = *reinterpret_cast<const uint4*>(at + c * kBlk);
              const uint32_t w4[4] = {raw[c].x, raw[c].y, raw[c].z, raw[c].w};
#pragma unroll
              for (int e = 0; e < 4; ++e) top = max(top, max((w4[e] << 16) & 0x7FFF0000u, w4[e] & 0x7FFF0000u));
            }
#pragma unroll
            for (int off = 4; off > 0; off >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, off));
            top >>= 23;                                             // its exponent
            // (subnormal rows as if it were 1; infinities and NaNs stay as they are)
            const int ex = top == 255u ? 127 : min(max((int)top, 1), 250);
            const float up = __uint_as_float((uint32_t)(254 - ex) << 23);   // 2^(127 - ex)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const uint32_t w4[4] = {raw[c].x, raw[c].y, raw[c].z, raw[c].w};
              uint32_t o[4];
#pragma unroll
              for (int e = 0; e < 4; ++e)
                o[e] = f16x2_rn(__uint_as_float(w4[e] << 16) * up, __uint_as_float(w4[e] & 0xFFFF0000u) * up);
              *reinterpret_cast<uint4*>(at + c * kBlk) = make_uint4(o[0], o[1], o[2], o[3]);
            }
            // (a factor of 0 would make a masked score's NaN, an infinite one that of a score of 0)
            if (l8 == 0)
              qscale[(it & 3) * kPM + q0 + 4 * q + g8] =
                  fminf(fmaxf(p.scale_log2 * __uint_as_float((uint32_t)ex << 23), 1.17549435e-38f), 3.40282347e+38f);
          }
        }
        landed(&bars.q_land);
        if (it > 0) ok = acquire(&bars.v_free, it - 1);  // the previous item's outputs have left V's slots
        if (!ok) break;
      }
      if (KV == GDA_KV_BF16) {
        const uint32_t sw[2] = {(uint32_t)(l8 ^ g8) << 4, (uint32_t)(l8 ^ (4 + g8)) << 4};
        const unsigned char* base = pool + (size_t)t.h * (2 * kD) + (is_v ? rank * kD : 0) + l8 * 16;
        const uint32_t pitch = (uint32_t)p.Hkv * (2 * kD);
#pragma unroll 1
        for (int j = t.ta; j < t.tb; ++j) {
          look_up(j + 2, n2);
          int sl[kPer];
#pragma unroll
          for (int x = 0; x < kPer; ++x) sl[x] = slot_of(n0[x], j, x), n0[x] = n1[x], n1[x] = n2[x];
          if (use > 0) ok = acquire(&empty[slot], use - 1);
          if (!ok) break;
          const uint32_t d0 = smem_u32(ring + slot * kHalf) + (row0 + g8) * 128;
          if (!PAIR || !is_v) {
#pragma unroll
            for (int q = 0; q < 8; ++q) {
              const int at = __shfl_sync(0xffffffffu, sl[0], 4 * q + g8);
              const unsigned char* src = base + (size_t)(uint32_t)max(at, 0) * pitch;
#pragma unroll
              for (int c = 0; c < 4; ++c) cp_async16(d0 + q * 512 + sw[q & 1] + c * kKBlk, src + 128 * c, at >= 0 ? 16 : 0);
            }
          } else {
#pragma unroll
            for (int q = 0; q < 16; ++q) {
              const int at = __shfl_sync(0xffffffffu, sl[(q >> 3) % kPer], (4 * q + g8) & 31);
              const unsigned char* src = base + (size_t)(uint32_t)max(at, 0) * pitch;
#pragma unroll
              for (int c = 0; c < 2; ++c) cp_async16(d0 + q * 512 + sw[q & 1] + c * kBlk, src + 128 * c, at >= 0 ? 16 : 0);
            }
          }
          landed(&land[slot]);
          if (++slot == slots) {
            slot = 0;
            ++use;
          }
        }
      } else {
        // codes.  A tile goes in kSubs steps per warp: copied (cp.async) into a small ring of the warp's own,
        // kStages steps ahead, and widened from there by the thread that copied it, 16 bytes at kU places.
        // The next tile's lines are sent to the L2 when its slots are known.
        // A place is four rows of 128 bytes (e4m3 K: half rows), or a 4-bit V's eight rows of 64.  The lanes
        // of a row's later parts take a neighbouring row's (sub_row), so that the eight 16-byte chunks that
        // are stored at a time lie in eight different banks
        auto gather = [&](auto of_v) {
          constexpr bool k8 = KV == GDA_KV_E4M3, kV = decltype(of_v)::value;   // (kV: half the dimensions of 128 keys)
          constexpr int kU = kPlaces, kSubs = k8 ? 4 : 2;
          // (a tile's steps unrolled: with their counts at run time the warps were bound by instructions, 64 x 4
          // tokens e4m3 113 us instead of 94, 48 single tokens over 4 bits 69.8 instead of 67.8.  Pairs over 4 bits,
          // whose softmax warps have more to do: unrolled 391 us, rolled 388)
          constexpr int kUnroll = k8 || !PAIR ? kSubs : 1;
          constexpr bool kHalves = k8 && !kV;                      // an e4m3 K row has two places
          constexpr int kPlaceRows = !k8 && kV ? 8 : 4;            // rows from one place to the next
          constexpr int kStepRows = (kHalves ? kU / 2 : kU) * kPlaceRows;
          static_assert(kStepRows % 8 == 0, "a row's swizzle does not depend on the step");
          const int part = !k8 && kV ? lane & 3 : l8;
          const int sub_row = k8 ? g8 ^ (l8 >> 2) : kV ? (lane >> 2) ^ (part & 2) : g8 ^ (l8 >> 1);
          auto row_of = [](int u) -> int { return kPlaceRows * (kHalves ? u >> 1 : u); };   // and sub_row
          const uint32_t pitch = (uint32_t)p.Hkv * (k8 ? kD : kCodeBytes), spitch = (uint32_t)p.Hkv * kScalePair;
          const unsigned char* base = pool + (size_t)t.h * (k8 ? kD : kCodeBytes) + (kV ? rank * (k8 ? 128 : 64) : 0) + part * 16;
          const unsigned char* sbase =
              k8 ? nullptr : p.scales + (size_t)t.h * kScalePair + (is_v ? kScaleBytes : 0) + (kV ? rank * 8 : 0) + ((part * 2) & ~3);
          unsigned char* stage = sm + Lay::kOffStage + (warp - kGatherWarp) * Lay::kStageWarp + lane * 16;
          const int c = k8 ? 2 * part : 4 * part;   // the first of a place's two (4 bits: four) 8-dimension chunks
          constexpr uint32_t kColBlk = kV ? kBlk : kKBlk;
          unsigned char* dst0 = ring + (row0 + sub_row) * 128 + (c >> 3) * kColBlk;
          const int sw[2] = {((c & 7) ^ (sub_row & 7)) << 4, ((c & 7) ^ ((4 + sub_row) & 7)) << 4};  // of rows 8 n, 8 n + 4
          int sl[kPer];        // the slots of the tile that is being copied, ij
          int ij = t.ta, islot = 0, wslot = 0;
          auto next_slots = [&](int* from) {
#pragma unroll
            for (int x = 0; x < kPer; ++x) sl[x] = slot_of(from[x], ij, x);
          };
          next_slots(n0);
          const uint32_t stage_to = smem_u32(stage);
          // step isub of tile ij into the staging ring
          auto copy = [&](int isub) {
            if (ij < t.tb) {
              const uint32_t to = stage_to + islot * Lay::kStageBytes;
              const int first = isub * kStepRows;   // (a step's rows lie in one of the two registers of slots)
              const int mine = first < 32 ? sl[0] : sl[kPer - 1];
              int at[kU];
#pragma unroll
              for (int u = 0; u < kU; ++u)
                at[u] = kHalves && (u & 1) ? at[u - 1] : __shfl_sync(0xffffffffu, mine, (first + row_of(u) + sub_row) & 31);
#pragma unroll
              for (int u = 0; u < kU; ++u) {
                const uint32_t o = (uint32_t)max(at[u], 0);
                cp_async16(to + u * 512, base + (size_t)o * pitch + (kHalves ? 128 * (u & 1) : 0), at[u] >= 0 ? 16 : 0);
                if (!k8)
                  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(to - lane * 12 + Lay::kStageCodes + u * 128),
                               "l"(sbase + (size_t)o * spitch), "r"(at[u] >= 0 ? 4 : 0) : "memory");
              }
              islot = islot + 1 == kStages ? 0 : islot + 1;
              if (isub == kSubs - 1) {
                ++ij;
                next_slots(n1);
#pragma unroll
                for (int x = 0; x < kPer; ++x) {
                  n1[x] = n2[x];
                  // the tile after next: to the L2, a row per lane
                  if (n1[x] >= 0 && (long long)n1[x] < p.num_slots) {
                    const unsigned char* line = base - part * 16 + (size_t)(uint32_t)n1[x] * pitch;
                    asm volatile("prefetch.global.L2 [%0];" ::"l"(line));
                    if (kHalves) asm volatile("prefetch.global.L2 [%0];" ::"l"(line + 128));
                  }
                }
                look_up(ij + 2, n2);
              }
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
          };
#pragma unroll 1
          for (int s = 0; s < kStages; ++s) copy(s % kSubs);
#pragma unroll 1
          for (int j = t.ta; j < t.tb; ++j) {
            if (use > 0) ok = acquire(&empty[slot], use - 1);
            if (!ok) break;
            unsigned char* dst = dst0 + slot * kHalf;
#pragma unroll kUnroll
            for (int sub = 0; sub < kSubs; ++sub) {
              asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
              const unsigned char* from = stage + wslot * Lay::kStageBytes;
              uint4 raw[kU];    // (all of the step's loads first)
              uint32_t s4[kU];
#pragma unroll
              for (int u = 0; u < kU; ++u) {
                raw[u] = *reinterpret_cast<const uint4*>(from + u * 512);
                if (!k8) s4[u] = *reinterpret_cast<const uint32_t*>(from - lane * 12 + Lay::kStageCodes + u * 128);
              }
#pragma unroll
              for (int u = 0; u < kU; ++u) {
                unsigned char* at = dst + (sub * kStepRows + row_of(u)) * 128 + (kHalves ? (u & 1) * 2 * kColBlk : 0);
                const int x7 = sw[(row_of(u) >> 2) & 1];
                if (k8) {
                  *reinterpret_cast<uint4*>(at + x7) = e4m3x8_to_f16(raw[u].x, raw[u].y);
                  *reinterpret_cast<uint4*>(at + (x7 ^ 16)) = e4m3x8_to_f16(raw[u].z, raw[u].w);
                } else {
                  const uint32_t f = e4m3x2_to_f16x2(s4[u] >> (16 * (part & 1)));
                  const uint32_t s_lo = __byte_perm(f, f, 0x1010), s_hi = __byte_perm(f, f, 0x3232);
                  *reinterpret_cast<uint4*>(at + x7) = e2m1x8_to_f16(raw[u].x, s_lo);
                  *reinterpret_cast<uint4*>(at + (x7 ^ 16)) = e2m1x8_to_f16(raw[u].y, s_lo);
                  *reinterpret_cast<uint4*>(at + (x7 ^ 32)) = e2m1x8_to_f16(raw[u].z, s_hi);
                  *reinterpret_cast<uint4*>(at + (x7 ^ 48)) = e2m1x8_to_f16(raw[u].w, s_hi);
                }
              }
              wslot = wslot + 1 == kStages ? 0 : wslot + 1;
              copy((sub + kStages) % kSubs);
            }
            landed(&land[slot]);
            if (++slot == slots) {
              slot = 0;
              ++use;
            }
          }
          cp_async_wait_all();
        };
        if (PAIR && is_v) gather(std::integral_constant<bool, PAIR>());
        else gather(std::false_type());
      }
      if (!ok) break;
      ++it;
    }
    cp_async_wait_all();
    if (!ok) fail();
  }

  // ---- teardown: every role of both CTAs is done (or gave up and waited for what it started)
  __syncwarp();
  tc_fence_before();
  if (PAIR) cluster_sync_all();
  else __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    if (PAIR) tmem_dealloc_pair(tmem, kTmemCols);
    else tmem_dealloc(tmem, kTmemCols);
  }
}

}  // namespace

template <int KV>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1) prefill_paged_kernel(const __grid_constant__ PagedParams p) {
  paged_body<KV, true>(p);
}
template <int KV>
__global__ void __launch_bounds__(kThreads, 1) prefill_paged_few_kernel(const __grid_constant__ PagedParams p) {
  paged_body<KV, false>(p);
}

// Joins the parts of the item that the start of share c = blockIdx.x + 1 cuts first:
//   m = max m_k, w_k = 2^(m_k - m), O = sum w_k O_k / (sum w_k l_k + sink)
// A thread has eight dimensions of a row, neighbouring threads neighbouring rows (as the parts are
// laid out).  Where an item has few rows and many parts, 2, 4 or 8 groups of a block's threads take
// a run of the parts each, and the first joins the runs.  Each in the order of the shares, and the
// groups a function of the counts: the same bits every time.  (One token
// at 8192 positions, whole call: 18.4 us, one group 46.7; at 131072 58 and 89.)
constexpr int kJoinThreads = 256, kJoinLog = 3, kJoinGroups = 1 << kJoinLog;
template <bool PAIR>
__global__ void __launch_bounds__(kJoinThreads) prefill_paged_join_kernel(const __grid_constant__ PagedParams p) {
  constexpr int kRowsI = Geo<PAIR>::kRows;
  __shared__ int part[kPagedMaxShares + 1];
  __shared__ int count[kJoinThreads / 32];
  __shared__ float runs[kJoinGroups - 1][11][kJoinThreads / kJoinGroups];   // (fewer groups: fewer runs of more threads)
  pdl_wait_prior_grid();
  pdl_launch_dependents();
  // (all that the cuts table has to say in one trip to memory; places past the last share end the table)
  const int c = blockIdx.x + 1, tid = threadIdx.x, shares = gridDim.x + 1;
  const int4 end = make_int4(p.B, 0, 0, 0);
  const int used = p.cuts[0].x;
  const int4 me = p.cuts[1 + c], before = p.cuts[c], seq = p.cuts[1 + shares + c];
  const int4 a = c + tid < shares ? p.cuts[1 + c + tid] : end, z = c + tid + 1 < shares ? p.cuts[2 + c + tid] : end;
  auto same = [&](const int4& x) { return x.x == me.x && x.y == me.y && x.z == me.z; };
  if (c >= used || me.x >= p.B || me.w == 0 || (same(before) && before.w > 0)) return;
  const int q0 = seq.x, flat0 = me.z * kRowsI;
  const int rows = min(kRowsI, seq.y * p.G - flat0);
  if ((int)(blockIdx.y * (kJoinThreads / kJoinGroups)) >= rows * (kD / 8)) return;
  // the parts: share c - 1's last one, then the first ones of the shares that start in the item; empty
  // shares are left out, the list in order by ballots
  int mine = -1;
  if (c + tid < used && same(a) && (c + tid + 1 >= used || !same(z) || z.w > a.w)) mine = 2 * (c + tid);
  const unsigned ball = __ballot_sync(0xffffffffu, mine >= 0);
  if ((tid & 31) == 0) count[tid >> 5] = __popc(ball);
  __syncthreads();
  int at = 1, parts = 1;
  for (int w = 0; w < kJoinThreads / 32; ++w) {
    if (w < (tid >> 5)) at += count[w];
    parts += count[w];
  }
  if (mine >= 0) part[at + __popc(ball & ((1u << (tid & 31)) - 1u))] = mine;
  if (tid == 0) part[0] = 2 * (c - 1) + 1;
  __syncthreads();
  // groups: as many as the blocks of a full item have threads for, four parts and more to each
  int lg = 0;   // log2 of their number
  while (lg < kJoinLog && (rows << (lg + 1)) <= kRowsI && parts > (4 << lg)) ++lg;
  const int pieces = kJoinThreads >> lg, group = tid / (kJoinThreads / kJoinGroups) >> (kJoinLog - lg), piece = tid & (pieces - 1);
  const int x = blockIdx.y * pieces + piece;
  if ((int)(blockIdx.y * pieces) >= rows * (kD / 8)) return;
  const bool in = x < rows * (kD / 8);
  const int c8 = in ? x / rows : 0, r = in ? x - c8 * rows : 0;
  const int tok = (int)((unsigned)(flat0 + r) / (unsigned)p.G), head = me.y * p.G + (flat0 + r - tok * p.G);
  uint4 g = make_uint4(0u, 0u, 0u, 0u);
  if (p.gate)
    g = __ldg(reinterpret_cast<const uint4*>(p.gate + (long long)(q0 + tok) * p.gate_stride + (long long)head * kD) + c8);
  // running max, so that a part's sums and values come in one trip
  float m = -INFINITY, l = 0.0f, e = 0.0f;
  float o[8] = {};
  auto add = [&](float pm, float pl, float pe, const float* po) {
    if (pl != 0.0f) {  // (0: no visible key in this part)
      const float top = fmaxf(m, pm), w = exp2f(pm - top), old = exp2f(m - top);
      m = top;
      l = l * old + w * pl;
      e = e * old + w * pe;
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i] = o[i] * old + w * po[i];
    }
  };
  const int k1 = (group + 1) * parts >> lg;
#pragma unroll 4
  for (int k = group * parts >> lg; k < k1; ++k) {
    const float4 s = __ldcg(p.part_ml + (size_t)part[k] * kRowsI + r);
    const float4* src = p.part_o + ((size_t)part[k] * 64 + 2 * c8) * kRowsI + r;
    const float4 u = __ldcg(src), v = __ldcg(src + kRowsI);
    const float po[8] = {u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
    add(s.x, s.y, s.z, po);
  }
  if (lg > 0) {
    float* run = &runs[0][0][0] + piece;   // [group - 1][value][piece]
    if (group > 0) {
      float* to = run + (group - 1) * 11 * pieces;
      to[0] = m, to[pieces] = l, to[2 * pieces] = e;
#pragma unroll
      for (int i = 0; i < 8; ++i) to[(3 + i) * pieces] = o[i];
    }
    __syncthreads();
    if (group > 0) return;
#pragma unroll 1
    for (int g1 = 0; g1 < (1 << lg) - 1; ++g1) {
      const float* from = run + g1 * 11 * pieces;
      float po[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) po[i] = from[(3 + i) * pieces];
      add(from[0], from[pieces], from[2 * pieces], po);
    }
  }
  if (!in) return;
  float wo = 1.0f;
  if (p.sinks) join_sink(p, head, m, l, e, wo);
  if (p.lse && c8 == 0) p.lse[(size_t)head * p.Tq + q0 + tok] = lse_of(m, e);
  const float inv = (l == 0.0f) ? 0.0f : wo * p.v_digits / l;
  const uint32_t keep = (l == 0.0f || wo == 0.0f) ? 0u : 0xFFFFFFFFu;
  uint32_t b[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) b[i] = bf16x2_rn(o[2 * i] * inv * p.v_power, o[2 * i + 1] * inv * p.v_power) & keep;
  if (p.gate) {
    uint32_t sg[4] = {g.x, g.y, g.z, g.w};
    sigmoids<1>(sg, p.table);
#pragma unroll
    for (int i = 0; i < 4; ++i) b[i] = mul_bf16x2(b[i], sg[i]);
  }
  reinterpret_cast<uint4*>(p.out + ((size_t)(q0 + tok) * p.Hq + head) * kD)[c8] = make_uint4(b[0], b[1], b[2], b[3]);
}

namespace {

// a programmatic dependent of the kernel before it
template <typename... Args>
cudaError_t launch(void (*kernel)(Args...), dim3 grid, int threads, uint32_t smem, cudaStream_t stream, const PagedParams& p) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}
template <bool PAIR>
cudaError_t launch_all(const PagedParams& p, int kv_dtype, int sms, cudaStream_t stream) {
  constexpr int kCtas = Geo<PAIR>::kCtas;
  const int shares = min(sms / kCtas, kPagedMaxShares / kCtas);
  if (shares < 1) return cudaErrorInvalidDevice;
  const dim3 grid((unsigned)(shares * kCtas));
  auto run = [&](auto kv) {
    constexpr int KV = decltype(kv)::value;
    return launch(PAIR ? prefill_paged_kernel<KV> : prefill_paged_few_kernel<KV>, grid, kThreads, Layout<KV>::kBytes, stream, p);
  };
  const cudaError_t e = kv_dtype == GDA_KV_BF16   ? run(std::integral_constant<int, GDA_KV_BF16>())
                        : kv_dtype == GDA_KV_E4M3 ? run(std::integral_constant<int, GDA_KV_E4M3>())
                                                  : run(std::integral_constant<int, GDA_KV_E2M1>());
  if (e != cudaSuccess || shares < 2) return e;
  const dim3 join((unsigned)(shares - 1), (unsigned)(Geo<PAIR>::kRows * (kD / 8) / kJoinThreads));
  return launch(prefill_paged_join_kernel<PAIR>, join, kJoinThreads, 0, stream, p);
}
template <int KV>
cudaError_t allow_smem() {
  const cudaError_t e = cudaFuncSetAttribute(prefill_paged_kernel<KV>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             (int)Layout<KV>::kBytes);
  if (e != cudaSuccess) return e;
  return cudaFuncSetAttribute(prefill_paged_few_kernel<KV>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Layout<KV>::kBytes);
}

}  // namespace

cudaError_t paged_init() {
  cudaError_t e = allow_smem<GDA_KV_BF16>();
  if (e == cudaSuccess) e = allow_smem<GDA_KV_E4M3>();
  if (e == cudaSuccess) e = allow_smem<GDA_KV_E2M1>();
  return e;
}

cudaError_t launch_prefill_paged(const PagedParams& params, int kv_dtype, cudaStream_t stream) {
  PagedParams p = params;
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  e = prefill_init(dev, stream);
  if (e == cudaSuccess) e = sigmoid_table(&p.table);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  const bool few = (long long)p.Tq * p.G <= (long long)kFewRows * p.B;
  return few ? launch_all<false>(p, kv_dtype, sms, stream) : launch_all<true>(p, kv_dtype, sms, stream);
}

}  // namespace gda
