// lora.h -- launchers of the low-rank adapter kernels (lora_few.cu,
// lora_shrink.cu, lora_expand.cu, lora_outer.cu) for the
// host API (lora.cu).  Not part of the public ABI.
#pragma once
#include <cuda_runtime.h>

#include <cstdint>


namespace wqmm {

// The rows in the order of their adapters.
struct LoraRows {
  const int* offsets;  // [adapters + 1]
  const int* source;   // [m]: row of every sorted place; behind offsets[adapters] the rows of no adapter
  int adapters;
  int64_t m;
};

// A matrix of m rows at a constant stride (elements).
struct LoraMat {
  const uint16_t* p;
  int64_t ld;
};

// low[p] = scale * x[source[p]] W^T, kept as two 16-bit numbers per value:
// low[p] = [hi (rp) | lo (rp)], value = factor[p] * (hi + lo).
struct LoraLow {
  uint16_t* low;   // [m][2 * rp]
  float* factor;   // [m] powers of two; float16 only
};

// One contraction over a long axis: k-major weights (adapters, rank, len) or
// rank-major ones (adapters, len, rank).
struct ShrinkParams {
  LoraMat x;
  const uint16_t* w;
  const float* scale;  // [adapters] or null
  LoraLow out;
  int len;
};

struct ExpandParams {
  LoraLow low;
  const uint16_t* w;   // (adapters, len, rank), or (adapters, rank, len) in the rank-major form
  LoraMat y;           // addend, p null: none
  uint16_t* out;
  int64_t ldo;
  int len;
  int bare;            // 1: the rows of no adapter are written too (y, or zeros)
};

struct OuterParams {
  LoraMat x;           // [m][len]
  LoraLow low;
  uint16_t* out;       // (adapters, rank, len) when rank_rows, else (adapters, len, rank)
  int len;
  int rank_rows;
};

int lora_padded_rank(int rank);
// Whether the gradients' kernels cut these rows into tiles of 16 instead of 128.
bool lora_few_rows(const LoraRows& rows, int rank);
// Whether a forward pass is launch_lora_few's one launch.
bool lora_one_launch(const LoraRows& rows, int rank, int bare, int sms);
// x by x k-major weights, and with count 2 then by rank-major ones.
cudaError_t launch_lora_shrink(const LoraRows& rows, const ShrinkParams* p, int count, int rank, bool bf16, int sms,
                               cudaStream_t s);
// Both contractions in one launch (sp.out and ep.low are not used).
cudaError_t launch_lora_few(const LoraRows& rows, const ShrinkParams& sp, const ExpandParams& ep, int rank, bool bf16,
                            int sms, cudaStream_t s);
cudaError_t launch_lora_expand(const LoraRows& rows, const ExpandParams& p, int rank, bool rank_major, bool bf16,
                               int sms, cudaStream_t s);
cudaError_t launch_lora_outer(const LoraRows& rows, const OuterParams (&p)[2], int rank, bool bf16, int sms,
                              cudaStream_t s);

}  // namespace wqmm
