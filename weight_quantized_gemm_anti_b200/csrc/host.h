// host.h -- host-side helpers of the C ABI shared by the operators' translation
// units: error messages, descriptor checks, and executors whose plan lives
// outside api.cu.  Not part of the public ABI.
#pragma once
#include <cuda_runtime.h>

#include <cstdint>
#include <memory>

#include "../../include/wqmm.h"

namespace wqmm {

// Record the calling thread's wqmm_last_error() message and return `code`.
__attribute__((format(printf, 2, 3))) wqmm_status fail(wqmm_status code, const char* fmt, ...);
// Clear the message and return WQMM_SUCCESS.
wqmm_status ok();
wqmm_status cuda_fail(cudaError_t e, const char* what);

const char* dt_name(int dt);
int dt_bytes(int dt);  // of an element; 0: not of whole bytes
int64_t numel(const wqmm_tensor* t);
bool contiguous(const wqmm_tensor* t);
bool aligned16(const void* p);
wqmm_status check_descriptor(const wqmm_tensor* t, const char* name);
int sm_count();
uint64_t round_up(uint64_t v, uint64_t a);

enum class OpKind { kWqmm, kQmm, kRoute, kLora };

// `rows` rows of `len` bytes, `ld` bytes from one to the next.
struct Memory {
  const char* name;
  const void* p;
  int64_t rows, len, ld;
  int may_be;  // of an input: the output (its number) that it may be itself, -1: none
};
Memory whole(const wqmm_tensor* t, const char* name, int may_be = -1);  // of a contiguous tensor

// The memory of an operator's tensors.  No output shares any with another tensor,
// except an input that is the output itself (same address, rows and stride) where it may be.
struct Memories {
  Memory out[3], in[8];
  int outs = 0, ins = 0;
  void add_out(const Memory& m) { out[outs++] = m; }
  void add_in(const Memory& m) { in[ins++] = m; }
};

// What phase 2 of an operator launches.  run() gets a workspace of at least
// the size phase 1 reported and launches on `s`.  `memories` is checked in phase 2, where the memory is used:
// phase 1 also answers for placeholder addresses, to a caller that wants the workspace's size.
struct OpPlan {
  Memories memories;
  virtual ~OpPlan() = default;
  virtual wqmm_status run(void* workspace, cudaStream_t s) = 0;
};

// Phase 1's end: hand out a one-shot executor holding `plan`.
wqmm_status hand_out(OpKind op, std::unique_ptr<OpPlan> plan, uint64_t workspace, uint64_t* workspace_size,
                     wqmm_executor** executor);
// Phase 2: check the executor and the workspace, run the plan, consume the executor.
wqmm_status run_plan(OpKind op, void* workspace, uint64_t workspace_size, wqmm_executor* executor,
                     wqmm_stream stream);

}  // namespace wqmm
