// gda_prefill_paged.h -- launch interface between the C ABI (gda_api.cu) and the attention of new
// tokens over a paged cache.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace gda {

struct PagedParams {
  const __nv_bfloat16* q;      // [Tq, Hq, 256], token t at t * q_stride elements
  const __nv_bfloat16* gate;   // likewise, or nullptr
  long long q_stride, gate_stride;
  const unsigned char* k_pool; // [num_slots, Hkv, row] of the cache's type
  const unsigned char* v_pool;
  const unsigned char* scales; // 4-bit: [num_slots, Hkv, 2, 16]
  long long num_slots;
  const int* cu_q;             // [B + 1] first new token of each sequence
  const int* indptr;           // [B + 1] first entry of `indices` of each sequence
  const int* indices;          // [nnz] slot of every position
  __nv_bfloat16* out;          // [Tq, Hq, 256]
  float* lse;                  // [Hq, Tq] natural log, or nullptr
  const float* sinks;          // [Hq] sink logits (natural units), or nullptr
  unsigned int* error;         // device error word
  int B, Tq, nnz, Hq, Hkv, G;
  int window, keep;            // window > 0: the last `window` positions and the first `keep`
  float scale_log2;            // scale * k_descale * log2(e)
  float v_digits, v_power;     // V's descale: 1 <= v_digits < 2 times a power of two (a sum may be 2^46 times that)
  long long wait_limit;
  const uint16_t* table;       // BF16 sigmoid of every BF16 code
  // workspace: where the shares of the work start, and what shares that cut an item leave of it
  int4* cuts;                  // {number of shares, -, -, -}, each share's start, each one's first sequence {row, tokens, -, -}
  float4* part_ml;             // [2 parts of a share][rows] {row max (log2), sum, unrounded sum, -}
  float4* part_o;              // [2 parts of a share][64][rows]: four dimensions of a row
};

constexpr int kPagedMaxShares = 160;  // CTAs, or twice as many as pairs of them
constexpr int kPagedRows = 128;       // rows of a part: one CTA's (a pair's part takes two)
// bytes of each part of the workspace
constexpr size_t kPagedCutBytes = 8192;
constexpr size_t kPagedMlBytes = (size_t)2 * kPagedMaxShares * kPagedRows * 16;
constexpr size_t kPagedOBytes = (size_t)2 * kPagedMaxShares * 64 * kPagedRows * 16;
static_assert((2 * kPagedMaxShares + 1) * 16 <= kPagedCutBytes, "cut table");

// kv_dtype: GDA_KV_* of the pools
cudaError_t launch_prefill_paged(const PagedParams& p, int kv_dtype, cudaStream_t stream);
cudaError_t paged_init();  // the kernels' attributes on the current device

}  // namespace gda
