// lora_shrink.cu -- the low-rank adapters' contractions over a long axis, low = scale * x W^T.
#include "lora_common.cuh"

namespace wqmm {
namespace {

// ------------------------------------------------------------------ shrink
// A CTA has BM rows and one of the cluster's shares of the contraction; the
// shares' sums meet in the cluster's shared memory, always in the order of the
// CTAs.  WM warps split the rows (16 each); with WM == 1 the four warps split
// the contraction's 16-wide steps instead.
template <int RT, bool KM, int BM>
struct ShrinkSmem {
  static constexpr int RP = RT * 16;
  static constexpr int kX = BM * 128;
  static constexpr int kWPitch = KM ? 128 : RP * 2 + 16;
  static constexpr int kW = KM ? RP * 128 : 64 * kWPitch;
  static constexpr int kStage = kX + kW;
  static constexpr int kStages = 4;
  static constexpr int kBytes = kStage * kStages;
};

// Few rows, k-major weights: nothing is shared between the warps, so the
// matrix instruction's operands come straight from global memory.  A thread
// loads 16 bytes of its rows and of its weight rows, eight neighbours of the
// contraction; four threads' 32 make two steps of the instruction.  Which
// element stands for which of a step's sixteen does not matter to the sum as
// long as both operands agree.  Each warp takes every fourth 32.
template <bool BF16, int RT>
__device__ __forceinline__ void few_rows_sum(const LoraRows& rows, const ShrinkParams& p, int rank, const Tile& tile,
                                             int k0, int k1, float (&acc)[RT * 2][4]) {
  constexpr int NT = RT * 2;
  constexpr int U = RT == 1 ? 4 : RT == 2 ? 2 : 1;  // 32s in flight: 16 to 18 loads
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, q = lane & 3;
  const uint16_t* x[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int64_t r = row_at(rows, tile.p0 + g + 8 * i, tile.p1);
    x[i] = r >= 0 ? p.x.p + r * p.x.ld + q * 8 : nullptr;
  }
  const uint16_t* w = p.w + (static_cast<int64_t>(tile.group) * rank + g) * p.len + q * 8;
  const uint4 zero = make_uint4(0, 0, 0, 0);
  for (int k = k0 + warp * 32; k < k1; k += 128 * U) {
    uint4 xv[U][2], wv[U][NT];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int at = k + u * 128;
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

template <bool BF16, int RT, bool KM, int WM>
__device__ __forceinline__ void shrink_tile(const LoraRows& rows, const ShrinkParams& p, int rank, int cs,
                                            const Tile& tile, uint8_t* sm) {
  constexpr int RP = RT * 16, NT = RT * 2, BM = WM * 16;
  using L = ShrinkSmem<RT, KM, BM>;
  constexpr int S = L::kStages;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t base = smem_u32(sm);
  const int crank = cs > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int steps_all = (p.len + 63) / 64;
  const int s0 = static_cast<int>(static_cast<int64_t>(steps_all) * crank / cs);
  const int s1 = static_cast<int>(static_cast<int64_t>(steps_all) * (crank + 1) / cs);
  float acc[NT][4];
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[n][i] = 0.f;
  const int wrow = WM == 1 ? 0 : warp * 16;
  if constexpr (WM == 1 && KM) {
    few_rows_sum<BF16, RT>(rows, p, rank, tile, s0 * 64, min(s1 * 64, p.len), acc);
  } else {
  const uint16_t* w = p.w + static_cast<int64_t>(tile.group) * rank * p.len;

  // this thread's rows of x: 16-byte chunk tid % 8 of rows tid / 8 + 16 i
  constexpr int XI = BM / 16;
  const int xc = tid & 7;
  const uint16_t* xrow[XI];
  bool xhas[XI];
#pragma unroll
  for (int i = 0; i < XI; ++i) {
    const int64_t r = row_at(rows, tile.p0 + tid / 8 + 16 * i, tile.p1);
    xhas[i] = r >= 0;
    xrow[i] = p.x.p + (r >= 0 ? r * p.x.ld : 0);
  }
  auto load = [&](int step, int stage) {
    const uint32_t xs = base + stage * L::kStage, ws = xs + L::kX;
    const int k = step * 64 + xc * 8;
#pragma unroll
    for (int i = 0; i < XI; ++i) {
      const int r = tid / 8 + 16 * i;
      const bool has = xhas[i] && k < p.len;
      cp16(xs + r * 128 + ((xc ^ (r & 7)) * 16), has ? xrow[i] + k : p.x.p, has);
    }
    if constexpr (KM) {
#pragma unroll
      for (int i = 0; i < RP / 16; ++i) {
        const int r = tid / 8 + 16 * i;
        const bool has = r < rank && k < p.len;
        cp16(ws + r * 128 + ((xc ^ (r & 7)) * 16), has ? w + static_cast<int64_t>(r) * p.len + k : w, has);
      }
    } else {
      constexpr int C = RP / 8;  // chunks of a row
#pragma unroll
      for (int i = 0; i < 64 * C / kThreads; ++i) {
        const int at = tid + i * kThreads, r = at / C, c = at % C, kk = step * 64 + r;
        const bool has = kk < p.len && c * 8 < rank;
        cp16(ws + r * L::kWPitch + c * 16, has ? w + static_cast<int64_t>(kk) * rank + c * 8 : w, has);
      }
    }
  };

#pragma unroll
  for (int i = 0; i < S - 1; ++i) {
    if (s0 + i < s1) load(s0 + i, i);
    cp_async_commit();
  }
  for (int st = s0; st < s1; ++st) {
    cp_async_wait_group<S - 2>();
    __syncthreads();
    if (st + S - 1 < s1) load(st + S - 1, (st - s0 + S - 1) % S);
    cp_async_commit();
    const uint32_t xs = base + ((st - s0) % S) * L::kStage, ws = xs + L::kX;
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) {
      if (WM == 1 && kk != warp) continue;
      uint32_t a[4];
      {
        const int r = wrow + (lane & 15), c = kk * 2 + (lane >> 4);
        ldsm4(a, xs + r * 128 + ((c ^ (r & 7)) * 16));
      }
#pragma unroll
      for (int n = 0; n < NT; n += 2) {
        uint32_t b[4];
        if constexpr (KM) {
          const int r = n * 8 + ((lane >> 4) << 3) + (lane & 7), c = kk * 2 + ((lane >> 3) & 1);
          ldsm4(b, ws + r * 128 + ((c ^ (r & 7)) * 16));
        } else {
          const int r = kk * 16 + (lane & 15), c = n + (lane >> 4);
          ldsm4t(b, ws + r * L::kWPitch + c * 16);
        }
        mma<BF16>(acc[n], a, b[0], b[1]);
        mma<BF16>(acc[n + 1], a, b[2], b[3]);
      }
    }
  }
  cp_async_wait_group<0>();
  __syncthreads();

  }

  // sums to shared memory, [row][RP]; with WM == 1 the warps' behind it first
  float* red = reinterpret_cast<float*>(sm);
  {
    float* mine = red + (WM == 1 ? (1 + warp) * 16 * RP : wrow * RP);
    const int g = lane >> 2, q = lane & 3;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      *reinterpret_cast<float2*>(mine + g * RP + n * 8 + 2 * q) = make_float2(acc[n][0], acc[n][1]);
      *reinterpret_cast<float2*>(mine + (g + 8) * RP + n * 8 + 2 * q) = make_float2(acc[n][2], acc[n][3]);
    }
  }
  if constexpr (WM == 1) {
    __syncthreads();
    for (int at = tid; at < 16 * RP; at += kThreads)
      red[at] = (red[16 * RP + at] + red[32 * RP + at]) + (red[48 * RP + at] + red[64 * RP + at]);
  }
  if (cs > 1)
    cluster_sync();
  else
    __syncthreads();

  // four values of a row per lane; the CTAs of the cluster share the rows
  constexpr int LANES = RP / 4, PER = kThreads / LANES;
  const int sub = tid % LANES;
  const float scale = p.scale ? p.scale[tile.group] : 1.f;
  for (int r0 = crank * PER; r0 < BM; r0 += cs * PER) {
    const int r = r0 + tid / LANES;
    const int64_t place = tile.p0 + r;
    const bool live = r < BM && place < tile.p1;
    float v[4] = {0.f, 0.f, 0.f, 0.f};
    if (live) {
      const uint32_t at = smem_u32(red + r * RP + sub * 4);
      float4 f[8];  // all CTAs' parts in flight at once
#pragma unroll
      for (int c = 0; c < 8; ++c)
        if (c < cs) f[c] = ld_cluster_f32x4(cs > 1 ? mapa_shared(at, c) : at);
#pragma unroll
      for (int c = 0; c < 8; ++c)
        if (c < cs) {
          v[0] += f[c].x;
          v[1] += f[c].y;
          v[2] += f[c].z;
          v[3] += f[c].w;
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] *= scale;
    if constexpr (!BF16) {
      // largest value of the row (NaN and infinities leave the factor at one)
      float top = 0.f;
      bool finite = true;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        top = fmaxf(top, fabsf(v[i]));
        finite = finite && isfinite(v[i]);
      }
      if (!finite) top = __int_as_float(0x7f800000);
#pragma unroll
      for (int d = 1; d < LANES; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
      // 2^14 <= top * up < 2^15: the exponent's complement, within the normal numbers
      float up = 1.f;
      if (top > 0.f && isfinite(top)) {
        const int e = static_cast<int>(__float_as_uint(top) >> 23);
        up = __uint_as_float(static_cast<uint32_t>(min(268 - e, 253)) << 23);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] *= up;
      if (live && sub == 0)
        p.out.factor[place] = __uint_as_float((254u << 23) - __float_as_uint(up));  // 1 / up, exactly
    }
    if (live) {
      uint32_t hi[2], lo[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float a = v[2 * i], b = v[2 * i + 1];
        hi[i] = Half<BF16>::put2(a, b);
        const float ha = Half<BF16>::get(hi[i] & 0xffff), hb = Half<BF16>::get(hi[i] >> 16);
        lo[i] = Half<BF16>::put2(isfinite(ha) ? a - ha : 0.f, isfinite(hb) ? b - hb : 0.f);
      }
      uint16_t* o = p.out.low + place * (2 * RP) + sub * 4;
      *reinterpret_cast<uint2*>(o) = make_uint2(hi[0], hi[1]);
      *reinterpret_cast<uint2*>(o + RP) = make_uint2(lo[0], lo[1]);
    }
  }
  if (cs > 1) cluster_sync();  // no CTA ends while another reads its sums
}

template <bool BF16, int RT, int WM, bool BOTH>
__global__ void __launch_bounds__(kThreads) shrink_kernel(LoraRows rows, ShrinkParams p0, ShrinkParams p1, int rank,
                                                          int cs) {
  extern __shared__ __align__(128) uint8_t sm[];
  pdl_wait();
  pdl_trigger();
  Tile tile;
  if (!find_tile(rows, 0, WM * 16, blockIdx.x / cs, tile)) return;  // the same for the whole cluster
  if (!BOTH || blockIdx.y == 0)
    shrink_tile<BF16, RT, true, WM>(rows, p0, rank, cs, tile, sm);
  else
    shrink_tile<BF16, RT, false, WM>(rows, p1, rank, cs, tile, sm);
}

template <bool BF16, int RT, int WM, bool BOTH>
cudaError_t shrink_as(const LoraRows& rows, const ShrinkParams* p, int rank, int sms, cudaStream_t s) {
  constexpr int BM = WM * 16;
  const int64_t tiles = most_tiles(rows.m, rows.adapters, BM);
  const int len = BOTH ? std::max(p[0].len, p[1].len) : p[0].len;
  // shares of the contraction: as many as fill the SMs four times over, each of at least four steps of 64
  int cs = 1;
  while (cs < 8 && tiles * (BOTH ? 2 : 1) * cs < 4 * sms && (len + 63) / 64 >= 8 * cs) cs *= 2;
  size_t smem = WM == 1 ? 0 : ShrinkSmem<RT, true, BM>::kBytes;
  if (BOTH) smem = std::max<size_t>(smem, ShrinkSmem<RT, false, BM>::kBytes);
  smem = std::max<size_t>(smem, static_cast<size_t>(WM == 1 ? 80 : BM) * RT * 16 * 4);
  auto kernel = shrink_kernel<BF16, RT, WM, BOTH>;
  if (const cudaError_t e = allow_smem(kernel, smem); e != cudaSuccess) return e;
  return launch_pdl(kernel, dim3(static_cast<unsigned>(tiles * cs), BOTH ? 2 : 1), dim3(kThreads), smem, cs, s, rows,
                    p[0], p[BOTH ? 1 : 0], rank, cs);
}

}  // namespace

int lora_padded_rank(int rank) { return 16 * padded_sixteenths(rank); }

cudaError_t launch_lora_shrink(const LoraRows& rows, const ShrinkParams* p, int count, int rank, bool bf16, int sms,
                               cudaStream_t s) {
  return with_rank(rank, [&](auto rt) {
    constexpr int RT = decltype(rt)::value;
    auto pick = [&](auto t, auto wm, auto both) {
      return shrink_as<decltype(t)::value, RT, decltype(wm)::value, decltype(both)::value>(rows, p, rank, sms, s);
    };
    auto by_wm = [&](auto t, auto both) {
      return few_rows(rows) ? pick(t, std::integral_constant<int, 1>(), both)
                            : pick(t, std::integral_constant<int, 4>(), both);
    };
    auto by_count = [&](auto t) {
      return count == 2 ? by_wm(t, std::true_type()) : by_wm(t, std::false_type());
    };
    return bf16 ? by_count(std::true_type()) : by_count(std::false_type());
  });
}

}  // namespace wqmm
