// lora_common.cuh -- what the kernels of the low-rank adapters share.  Low-rank adapters of
// many requests beside a shared projection, and their gradients:
//
//   forward   low = s x A^T          (shrink: contraction over k)
//             out = y + low B^T      (expand: contraction over the rank)
//   backward  back = s g B           (shrink over n),  low again from x
//             dx = dx0 + back A      (expand)
//             dA = back^T x, dB = g^T low   (outer: contraction over the rows)
//
// with A, B and s those of the row's adapter.  The rows are read in the order
// of their adapters (`source`), so that a tile of rows shares one adapter.
//
// The rank is small, so a row's 2 * rank * len products cost little beside its
// bytes: memory bounds all three kernels.  low and back are sums over a long
// axis and the next product's input; they are kept as two 16-bit numbers (the
// value's rounding and the rounding of what is left), 16 (bfloat16) or 22
// (float16) bits of it, so that they cost no accuracy beside a 16-bit result
// while both products run on the 16-bit matrix instructions.  float16's
// exponents do not reach as far as 32-bit ones: a row of low is first scaled
// by a power of two that puts its largest value just below the type's largest.
// The contraction over the rows, which has one such power for all of them, keeps 2^-38 of the
// adapter's largest value (the type's smallest number beside 2^14).
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <type_traits>

#include "internal.h"
#include "launch.cuh"
#include "lora.h"
#include "ptx.cuh"

namespace wqmm {
namespace {

constexpr int kThreads = 128;
// The power of two of a float16 row of low that has no finite value but zero: below those of all others.
constexpr float kNoValue = 0x1p-127f;

// ------------------------------------------------------------------ types
template <bool BF16>
struct Half;
template <>
struct Half<true> {
  static __device__ __forceinline__ float get(uint16_t v) { return __uint_as_float(static_cast<uint32_t>(v) << 16); }
  static __device__ __forceinline__ uint32_t put2(float a, float b) {
    __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<uint32_t*>(&h);
  }
};
template <>
struct Half<false> {
  static __device__ __forceinline__ float get(uint16_t v) { return __half2float(__ushort_as_half(v)); }
  static __device__ __forceinline__ uint32_t put2(float a, float b) {
    __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<uint32_t*>(&h);
  }
};

// d += a b: 16 x 8 x 16, 16-bit inputs, 32-bit sums.
template <bool BF16>
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (BF16)
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool has) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(has ? 16 : 0) : "memory");
}
__device__ __forceinline__ void st_cluster_f32x4(uint32_t addr, float a, float b, float c, float d) {
  asm volatile("st.shared::cluster.v4.f32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "f"(a), "f"(b), "f"(c), "f"(d) : "memory");
}
// ------------------------------------------------------------------ tiles of rows
// Tile t of the sorted rows when every group of rows is cut into tiles of `bm`:
// its group and its rows [p0, p1).  The groups are the adapters and, with
// `bare`, the rows of none behind them.  The offsets are clamped to [0, m], so
// that no value of theirs leads out of the tensors.  Called by whole warps.
struct Tile {
  int group, p0, p1;
};
__device__ __forceinline__ int offset_at(const LoraRows& r, int g) {
  const int m = static_cast<int>(r.m);
  return g > r.adapters ? m : min(max(r.offsets[g], 0), m);
}
__device__ __forceinline__ bool find_tile(const LoraRows& r, int bare, int bm, int t, Tile& out) {
  const int lane = threadIdx.x & 31;
  const int groups = r.adapters + bare;
  for (int g0 = 0; g0 < groups; g0 += 32) {
    const int g = g0 + lane;
    int lo = 0, hi = 0;
    if (g < groups) {
      lo = offset_at(r, g);
      hi = offset_at(r, g + 1);
    }
    const int n = hi > lo ? (hi - lo - 1) / bm + 1 : 0;
    int upto = n;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, upto, d);
      if (lane >= d) upto += v;
    }
    const int all = __shfl_sync(0xffffffffu, upto, 31);
    if (t < all) {
      const int at = __popc(__ballot_sync(0xffffffffu, upto <= t));
      const int first = __shfl_sync(0xffffffffu, upto - n, at);
      out.group = g0 + at;
      out.p1 = __shfl_sync(0xffffffffu, hi, at);
      out.p0 = __shfl_sync(0xffffffffu, lo, at) + (t - first) * bm;
      if (out.p1 - out.p0 > bm) out.p1 = out.p0 + bm;
      return true;
    }
    t -= all;
  }
  return false;
}
// Row of a sorted place, -1 behind the tile (or where the order names no row).
__device__ __forceinline__ int row_at(const LoraRows& r, int p, int p1) {
  if (p >= p1) return -1;
  const int v = r.source[p];
  return v < r.m ? v : -1;
}
// Most tiles that m rows in `groups` groups can make.
int64_t most_tiles(int64_t m, int groups, int bm) {
  const int64_t g = std::min<int64_t>(groups, m);
  return (m + g * (bm - 1)) / bm;
}

__host__ __device__ constexpr int padded_sixteenths(int rank) {
  return rank <= 16 ? 1 : rank <= 32 ? 2 : rank <= 64 ? 4 : 8;
}

// ------------------------------------------------------------------ launches
// Calls f with the padded rank's sixteenth (1, 2, 4 or 8) as a constant.
template <typename F>
cudaError_t with_rank(int rank, F&& f) {
  switch (padded_sixteenths(rank)) {
    case 1: return f(std::integral_constant<int, 1>());
    case 2: return f(std::integral_constant<int, 2>());
    case 4: return f(std::integral_constant<int, 4>());
    default: return f(std::integral_constant<int, 8>());
  }
}

// Whether a gradient's rows are cut into tiles of 16 instead of 128: few rows, or
// few per adapter, and the fewer the larger the rank: at 128 the sums of 16
// rows do not leave the registers enough loads under way.  k = n = 4096 (k = 1024,
// n = 8192 favours the small tiles, the reverse the large ones), the adapters'
// whole gradient, tiles of 16 and of 128 rows, in us:
//   one adapter   rank 16    64 rows 10.3, 13.5  256 rows 14.4, 17.0  512 rows 19.8, 19.6
//                 rank 64    64 rows 18.6, 20.0  128 rows 21.6, 20.7  256 rows 26.0, 24.6
//                 rank 128    4 rows 18.0, 25.0   64 rows 21.4, 25.7  128 rows 29.1, 26.4
//   32 adapters   rank 16    64 rows 20.4, 29.2  512 rows 25.1, 36.4  1000 rows 30.3, 37.1
//                 rank 64    64 rows 43.9, 52.9  512 rows 57.1, 61.3
//                 rank 128    4 rows 70.3, 76.2   64 rows 116, 112    512 rows 157, 130
bool few_rows(const LoraRows& r, int rank) {
  if (rank > 64) return r.m <= 64;
  return r.m <= (rank <= 32 ? 256 : 128) || r.m <= 16 * static_cast<int64_t>(r.adapters);
}

}  // namespace
}  // namespace wqmm
