// lora_tc.cuh -- what the adapters' tcgen05 kernels (lora_shrink.cu,
// lora_expand.cu, lora_outer.cu) share: shared-memory operands of both majors and
// the copies that fill them.
//
// The rows of a tile lie anywhere in x (the order of the adapters), so they are
// copied by four warps with 16-byte asynchronous copies, 128 to 256
// neighbouring bytes of a row by the lanes next to each other; a gathering
// tensor copy (four rows of 128 bytes each) moved 7 bytes per clock and SM
// where 23 are wanted.  A stage's barrier counts the copies as they land.
#pragma once
#include "lora_common.cuh"

namespace wqmm {
namespace {

constexpr int kCopyThreads = 128;  // warps 0 to 3

// D[tmem] (+)= A[smem] * B[smem]^T, kind::f16.
__device__ __forceinline__ void mma_f16_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}

// An operand in shared memory.  Rows of `row_bytes` (32, 64 or 128) in the
// swizzle of that width; `sbo` bytes from eight rows to the next eight; for the
// operand whose rows run along the contraction (MN-major) `lbo` bytes from one
// row_bytes-wide block of it to the next.
__host__ __device__ constexpr uint64_t operand_bits(int row_bytes, uint32_t lbo, uint32_t sbo) {
  return (static_cast<uint64_t>(lbo >> 4) << 16) | (static_cast<uint64_t>(sbo >> 4) << 32) | (1ull << 46) |
         (static_cast<uint64_t>(row_bytes == 128 ? 2 : row_bytes == 64 ? 4 : 6) << 61);
}
__device__ __forceinline__ uint64_t operand(uint32_t addr, uint64_t bits) { return bits | ((addr & 0x3FFFFu) >> 4); }

constexpr uint32_t kAMn = 1u << 15, kBMn = 1u << 16;  // instruction descriptor: operand is MN-major

// Byte of 16-byte chunk c of row r where rows of ROW bytes are swizzled.
template <int ROW>
__device__ __forceinline__ uint32_t swizzled(int r, int c) {
  return r * ROW + ((c ^ (ROW == 128 ? r & 7 : ROW == 64 ? (r >> 1) & 3 : (r >> 2) & 1)) * 16);
}

// A rank-wide operand: 64 rows along the contraction (MN-major) of RP columns,
// in blocks of up to 64 columns.
template <int RT>
struct RankRows {
  static constexpr int RP = RT * 16;
  static constexpr int kCols = RP < 64 ? RP : 64;  // of one block
  static constexpr int kRow = kCols * 2;
  static constexpr int kBlock = 64 * kRow;
  static constexpr int kBytes = RP / kCols * kBlock;
  static constexpr uint64_t kBits = operand_bits(kRow, RP > kCols ? kBlock : 16, 8 * kRow);
  static constexpr uint32_t kStep = 16 * kRow;  // bytes from one MMA's sixteen rows to the next
  // byte of columns 8 c .. 8 c + 7 of row r
  static __device__ __forceinline__ uint32_t at(int r, int c) {
    constexpr int C = kCols / 8;
    return c / C * kBlock + swizzled<kRow>(r, c % C);
  }
};

__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort, uint32_t* err,
                                          uint32_t code) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort, err, code));
}

// A copying warp hands a stage over without waiting for its copies: the barrier
// counts them when they land.
__device__ __forceinline__ void hand_over(uint64_t* full) {
  cp_async_mbar_arrive(full);
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(full);
}
__device__ __forceinline__ void copies_landed() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// The MMA warp's wait for a stage.  What threads have written to shared memory
// becomes visible to the tensor core by the fence; the waiting side makes it,
// since a copying thread's would wait for all its copies under way.
__device__ __forceinline__ bool stage_wait(uint64_t* full, uint32_t parity, volatile int* abort, uint32_t* err) {
  if (!warp_wait(full, parity, abort, err, kDevTimeoutMma)) return false;
  fence_proxy_async_smem();
  tc_fence_after();
  return true;
}

}  // namespace
}  // namespace wqmm
