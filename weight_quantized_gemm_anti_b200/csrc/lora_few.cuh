// lora_few.cuh -- tiles of 16 rows of the low-rank adapters: their contraction
// (lora_few.cu, lora_shrink.cu), and a row's two 16-bit numbers.
#pragma once
#include "lora_common.cuh"

namespace wqmm {
namespace {

// Four neighbours of a row of low (LANES lanes have the row) times `scale`, as
// two 16-bit numbers each.  float16: the row is first brought to where its
// largest finite value is below 2^15 by a power of two, whose inverse is returned.  A row without one
// (a masked token's zeros) returns kNoValue: its factor must not be the largest of its adapter's rows, to
// which the weights' gradients bring them all.  Values that are not finite stay so under any power; beside
// them the row's others keep their bits.
template <bool BF16, int LANES>
__device__ __forceinline__ float split_row(float (&v)[4], float scale, uint2& hi, uint2& lo) {
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] *= scale;
  float up = 1.f;
  bool has = true;
  if constexpr (!BF16) {
    // the row's largest value, NaN and infinities aside
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) top = fmaxf(top, isfinite(v[i]) ? fabsf(v[i]) : 0.f);
#pragma unroll
    for (int d = 1; d < LANES; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
    has = top > 0.f;
    // 2^14 <= top * up < 2^15: the exponent's complement, within the normal numbers
    const int e = static_cast<int>(__float_as_uint(top) >> 23);
    up = __uint_as_float(static_cast<uint32_t>(min(268 - e, 253)) << 23);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] *= up;
  }
  uint32_t h[2], l[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float a = v[2 * i], b = v[2 * i + 1];
    h[i] = Half<BF16>::put2(a, b);
    const float ha = Half<BF16>::get(h[i] & 0xffff), hb = Half<BF16>::get(h[i] >> 16);
    l[i] = Half<BF16>::put2(isfinite(ha) ? a - ha : 0.f, isfinite(hb) ? b - hb : 0.f);
  }
  hi = make_uint2(h[0], h[1]);
  lo = make_uint2(l[0], l[1]);
  return has ? __uint_as_float((254u << 23) - __float_as_uint(up)) : kNoValue;  // 1 / up, exactly
}

// Four neighbours of the sum of NW warps' parts, `stride` floats apart.
template <int NW>
__device__ __forceinline__ float4 sum_of_warps(const float* part, int stride) {
  float4 v[NW];
#pragma unroll
  for (int w = 0; w < NW; ++w) v[w] = *reinterpret_cast<const float4*>(part + w * stride);
#pragma unroll
  for (int h = NW / 2; h > 0; h /= 2)
#pragma unroll
    for (int w = 0; w < h; ++w) {
      v[w].x += v[w + h].x;
      v[w].y += v[w + h].y;
      v[w].z += v[w + h].z;
      v[w].w += v[w + h].w;
    }
  return v[0];
}

// The contraction of k-major weights with a tile of 16 rows, NW warps sharing it.
// Nothing is shared between the warps, so the matrix instruction's operands come straight from global memory.  A thread
// loads 16 bytes of its rows and of its weight rows, eight neighbours of the
// contraction; four threads' 32 make two steps of the instruction.  Which
// element stands for which of a step's sixteen does not matter to the sum as
// long as both operands agree.  Each warp takes every NW-th 32.
template <bool BF16, int RT, int NW>
__device__ __forceinline__ void few_rows_sum(const LoraRows& rows, const ShrinkParams& p, int rank, const Tile& tile,
                                             int k0, int k1, float (&acc)[RT * 2][4]) {
  constexpr int NT = RT * 2;
  // 32s in flight: 10 to 20 loads (rank 64 in eight warps, 1000 rows of 4096: two 15.1 us, one 16.1; rank 32 three:
  // 3 % slower)
  constexpr int U = RT == 1 ? 4 : RT == 2 || (RT == 4 && NW == 8) ? 2 : 1;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, q = lane & 3;
  const uint16_t* x[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r = row_at(rows, tile.p0 + g + 8 * i, tile.p1);
    x[i] = r >= 0 ? p.x.p + r * p.x.ld + q * 8 : nullptr;
  }
  const uint16_t* w = p.w + (static_cast<int64_t>(tile.group) * rank + g) * p.len + q * 8;
  const uint4 zero = make_uint4(0, 0, 0, 0);
  for (int k = k0 + warp * 32; k < k1; k += 32 * NW * U) {
    uint4 xv[U][2], wv[U][NT];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int at = k + u * 32 * NW;
      const bool in = at < k1;
#pragma unroll
      for (int n = 0; n < NT; ++n)
        wv[u][n] = in && n * 8 < rank
                       ? *reinterpret_cast<const uint4*>(w + static_cast<int64_t>(n) * 8 * p.len + at) : zero;
#pragma unroll
      for (int i = 0; i < 2; ++i) xv[u][i] = in && x[i] ? *reinterpret_cast<const uint4*>(x[i] + at) : zero;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t a0[4] = {xv[u][0].x, xv[u][1].x, xv[u][0].y, xv[u][1].y};
      const uint32_t a1[4] = {xv[u][0].z, xv[u][1].z, xv[u][0].w, xv[u][1].w};
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        mma<BF16>(acc[n], a0, wv[u][n].x, wv[u][n].y);
        mma<BF16>(acc[n], a1, wv[u][n].z, wv[u][n].w);
      }
    }
  }
}

}  // namespace
}  // namespace wqmm
