// route.h -- launchers of the token routing kernels (kernels_route.cu) for the
// host API (route.cu).  Not part of the public ABI.
#pragma once
#include <cuda_runtime.h>

#include <cstdint>

namespace wqmm {

constexpr int kMaxGroups = 2048;  // experts, or adapters

// Element type of activations and weights inside the routing kernels.
enum RouteType : int { kRtF16 = 0, kRtBf16 = 1, kRtF32 = 2 };

struct SortParams {
  const void* ids;    // [slots] int32 or int64
  int ids64;
  int64_t slots;
  int groups;
  int chunk;          // slots of one CTA
  int chunks;         // CTAs; > 1: hist holds [chunks][groups + 1] counts
  int* hist;
  int* offsets;       // [groups + 1]
  int* source;        // [slots]
  int* position;      // [slots]
};

struct DispatchParams {
  const uint8_t* x;        // [tokens][row_bytes]
  uint8_t* out;            // [rows][row_bytes]
  const int* position;     // [tokens][top]
  int64_t tokens, rows, row_bytes;
  int top;
};

struct CombineParams {
  const void* x_sorted;    // [rows][hidden]
  const int* position;     // [tokens][top]
  const void* weights;     // [tokens][top], or null: all one
  const void* x3;          // [tokens][hidden], or null
  void* out;               // [tokens][hidden]
  int64_t tokens, rows, hidden;
  int top;
  int type, wtype;         // RouteType
};

struct CombineGradParams {
  const void* grad;        // [tokens][hidden]
  const void* x_sorted;    // [rows][hidden]
  const int* position;     // [tokens][top]
  const void* weights;     // [tokens][top]
  void* grad_sorted;       // [rows][hidden]
  void* grad_weights;      // [tokens][top]
  int64_t tokens, rows, hidden;
  int top;
  int type, wtype;
};

// Fills chunk and chunks; returns the bytes of hist (0: none).
uint64_t plan_sort(SortParams& p);
cudaError_t launch_sort(const SortParams& p, cudaStream_t s);
cudaError_t launch_dispatch(const DispatchParams& p, cudaStream_t s);
cudaError_t launch_combine(const CombineParams& p, cudaStream_t s);
cudaError_t launch_combine_grad(const CombineGradParams& p, cudaStream_t s);

}  // namespace wqmm
