// gda_prefill.h -- launch interface between the C ABI (gda_api.cu) and the prefill kernel.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace gda {

struct PrefillParams {
  __nv_bfloat16* out;          // [B, Sq, Hq, D]
  float* lse;                  // [B, Hq, Sq] natural log, or nullptr
  const __nv_bfloat16* gate;   // [B, Sq, Hq, D] (read directly only for rows with no visible key)
  const int* kv_lens;          // [B] or nullptr (all Skv)
  unsigned int* error;         // device error word (kErr* bits)
  int B, Sq, Skv, Hq, Hkv;
  float scale_log2;            // scale * log2(e)
  int causal;
  int fuse_gate;
  long long wait_limit;        // SM cycles after which a pipeline wait gives up (kWaitLimitCycles;
                               // shorter only in the failure-path test)
  // packed form (one [T, H, D] tensor each, B sequences): Sq and Skv are the tensors' rows
  const int* cu_q = nullptr;   // [B + 1] first query row of each sequence
  const int* cu_k = nullptr;   // [B + 1] first key row
  long long gate_stride = 0;   // elements between the gate's tokens
  const uint16_t* table = nullptr;  // BF16 sigmoid of every BF16 code
};

// The most 128-row query blocks that B sequences of `rows` rows in all can have.
inline long long packed_blocks(long long rows, long long B) {
  const long long n = rows / 128 + B;  // each sequence ends at most one block early
  return n < rows ? n : rows;
}

// Prefill / extend gated SDPA (tcgen05); q, k, v, gate are [B, S, H, 256] BF16.
cudaError_t launch_prefill(const PrefillParams& p, const void* q, const void* k, const void* v, const void* gate,
                           cudaStream_t stream);

// Parts that the padded and the packed kernel share (gda_prefill.cu): the tensor map of a
// [B, S, H, 256] BF16 tensor with box {64, rows, blocks}, the first use on a device (both
// kernels' attributes, the sigmoid table), and the table's address on the current device.
bool make_map_kv(CUtensorMap* m, const void* base, int B, int S, int H, int rows, int blocks, int64_t pitch);
cudaError_t prefill_init(int dev, cudaStream_t stream);
cudaError_t sigmoid_table(const uint16_t** table);
cudaError_t packed_init();  // gda_prefill_packed.cu

// The same over packed sequences; pitches are elements between tokens.
cudaError_t launch_prefill_packed(const PrefillParams& p, const void* q, int64_t q_pitch, const void* k,
                                  int64_t k_pitch, const void* v, int64_t v_pitch, const void* gate,
                                  cudaStream_t stream);

}  // namespace gda
