// lora_tc.cuh -- what the adapters' tcgen05 kernels (lora_shrink.cu,
// lora_outer.cu) share: gathered tensor copies, shared-memory operand
// descriptors for both majors, and tensor map shapes.
#pragma once
#include "lora_common.cuh"

namespace wqmm {
namespace {

constexpr int kTcThreads = 192;  // copy warp, MMA warp, four warps for the rest

// Four rows of a tensor map whose box is one row of 64 columns: row i of the
// four at dst + 128 i (128-byte swizzle).  A row outside the tensor reads as zeros.
__device__ __forceinline__ void tma_gather4(uint32_t dst, const CUtensorMap* map, uint64_t* bar, int32_t col, int4 r) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, "
      "%5, %6, %7}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(col), "r"(r.x), "r"(r.y), "r"(r.z), "r"(r.w)
      : "memory");
}

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, uint64_t* bar, int32_t c0, int32_t c1,
                                            int32_t c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], "
      "[%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2)
      : "memory");
}

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

// A rank-wide operand (RP columns, 64 rows along the contraction, MN-major):
// bytes of a row of one block, of the whole, and its descriptor.
template <int RT>
struct RankRows {
  static constexpr int RP = RT * 16;
  static constexpr int kCols = RP < 64 ? RP : 64;  // columns of one block (one tensor copy)
  static constexpr int kBlocks = RP / kCols;
  static constexpr int kRow = kCols * 2;
  static constexpr int kBlock = 64 * kRow;
  static constexpr int kBytes = kBlocks * kBlock;
  static constexpr uint64_t kBits = operand_bits(kRow, kBlocks > 1 ? kBlock : 16, 8 * kRow);
  static constexpr uint32_t kStep = 16 * kRow;  // bytes from one MMA's sixteen rows to the next
};

// Both contractions' tensor maps.
struct TcMaps {
  CUtensorMap x[2];  // gathered rows: box 64 columns x 1 row, 128-byte swizzle
  CUtensorMap w[2];
};

__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort, uint32_t* err,
                                          uint32_t code) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort, err, code));
}

}  // namespace
}  // namespace wqmm
