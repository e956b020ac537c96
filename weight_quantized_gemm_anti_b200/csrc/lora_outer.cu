// lora_outer.cu -- the gradients of the low-rank adapters' weights, contractions over the rows.
#include "lora_common.cuh"

namespace wqmm {
namespace {

// ------------------------------------------------------------------ outer
// A CTA has 128 columns of one adapter's gradient and one of the cluster's
// shares of the adapter's rows; the shares meet as the shrink's do.  The
// instruction's rows are the columns of x, its columns the rank; four warps
// have 32 columns each.  An adapter without rows gets zeros.
template <int RT>
struct OuterSmem {
  static constexpr int RP = RT * 16;
  static constexpr int kXPitch = 256 + 16, kLPitch = RP * 4 + 16;
  static constexpr int kX = 64 * kXPitch, kL = 64 * kLPitch;
  static constexpr int kStage = kX + kL + 256;
  static constexpr int kStages = 3;
  static constexpr int kBytes = kStage * kStages;
  static constexpr int kRedPitch = RP + 1;
  static_assert(128 * kRedPitch * 4 <= kBytes, "the sums reuse the stages");
};

template <bool BF16, int RT>
__global__ void __launch_bounds__(kThreads) outer_kernel(LoraRows rows, OuterParams p0, OuterParams p1, int rank,
                                                         int cs, int tiles0) {
  extern __shared__ __align__(128) uint8_t sm[];
  __shared__ float tops[4];
  constexpr int RP = RT * 16, NT = RT * 2;
  using L = OuterSmem<RT>;
  constexpr int S = L::kStages;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t base = smem_u32(sm);
  const int crank = cs > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int ct = blockIdx.x / cs;
  const OuterParams& p = ct < tiles0 ? p0 : p1;
  const int c0 = (ct < tiles0 ? ct : ct - tiles0) * 128;
  const int adapter = blockIdx.y;
  const int64_t lo = offset_at(rows, adapter), hi = max(offset_at(rows, adapter + 1), lo);
  const int64_t steps = (hi - lo + 63) / 64;
  const int64_t s0 = steps * crank / cs, s1 = steps * (crank + 1) / cs;

  // this thread's rows of x in a step: 16-byte chunk tid % 16 of rows tid / 16 + 8 i.  Their numbers are
  // loaded a step before the rows are.
  const int xc = tid & 15;
  const bool in = c0 + xc * 8 < p.len;
  int64_t next[8];
  auto find = [&](int64_t step) {
#pragma unroll
    for (int i = 0; i < 8; ++i) next[i] = step < s1 ? row_at(rows, lo + step * 64 + tid / 16 + 8 * i, hi) : -1;
  };
  auto load_x = [&](int stage) {
    const uint32_t xs = base + stage * L::kStage;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int r = tid / 16 + 8 * i;
      const bool has = in && next[i] >= 0;
      cp16(xs + r * L::kXPitch + xc * 16, has ? p.x.p + next[i] * p.x.ld + c0 + xc * 8 : p.x.p, has);
    }
  };
  auto load_low = [&](int64_t step, int stage) {
    const uint32_t ls = base + stage * L::kStage + L::kX, fs = ls + L::kL;
    const int64_t r0 = lo + step * 64;
    constexpr int C = RP / 4;  // 16-byte chunks of a row of low
#pragma unroll
    for (int i = 0; i < 64 * C / kThreads; ++i) {
      const int at = tid + i * kThreads, r = at / C, cc = at % C;
      const bool has = r0 + r < hi;
      cp16(ls + r * L::kLPitch + cc * 16, has ? p.low.low + (r0 + r) * (2 * RP) + cc * 8 : p.low.low, has);
    }
    if (!BF16 && tid < 64) {
      const bool has = r0 + tid < hi;
      cp4(fs + tid * 4, has ? p.low.factor + r0 + tid : p.low.factor, has);
    }
  };
  // x and the order are older than the launch before this one, which has waited for all that
  // came before it: they are read while it ends, low after that
#pragma unroll
  for (int i = 0; i < S - 1; ++i) {
    find(s0 + i);
    if (s0 + i < s1) load_x(i);
  }
  find(s0 + S - 1);
  pdl_wait();
  pdl_trigger();
#pragma unroll
  for (int i = 0; i < S - 1; ++i) {
    if (s0 + i < s1) load_low(s0 + i, i);
    cp_async_commit();
  }

  // the largest factor of this CTA's rows: the others' low values are scaled to it
  float top = 1.f, below = 1.f;
  if constexpr (!BF16) {
    top = 0.f;
    for (int64_t r = lo + s0 * 64 + tid; r < min(lo + s1 * 64, hi); r += kThreads) top = fmaxf(top, p.low.factor[r]);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
    if (lane == 0) tops[warp] = top;
    __syncthreads();
    top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]));
    if (!(top > 0.f)) top = 1.f;  // no rows
    below = 1.f / top;            // of a power of two: exact
  }

  float acc[2][NT][4];
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[m][n][i] = 0.f;

  for (int64_t st = s0; st < s1; ++st) {
    cp_async_wait_group<S - 2>();
    __syncthreads();
    if (st + S - 1 < s1) {
      const int stage = static_cast<int>((st - s0 + S - 1) % S);
      load_x(stage);
      load_low(st + S - 1, stage);
    }
    cp_async_commit();
    find(st + S);
    const uint32_t xs = base + static_cast<int>((st - s0) % S) * L::kStage, ls = xs + L::kX;
    const float* fs = reinterpret_cast<const float*>(sm + static_cast<int>((st - s0) % S) * L::kStage + L::kX + L::kL);
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) {
      uint32_t a[2][4];
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        const int r = kk * 16 + ((lane >> 4) << 3) + (lane & 7), c = warp * 4 + m * 2 + ((lane >> 3) & 1);
        ldsm4t(a[m], xs + r * L::kXPitch + c * 16);
      }
      __half2 f0, f1;
      if constexpr (!BF16) {
        const int r = kk * 16 + 2 * (lane & 3);
        f0 = __floats2half2_rn(fs[r] * below, fs[r + 1] * below);
        f1 = __floats2half2_rn(fs[r + 8] * below, fs[r + 9] * below);
      }
#pragma unroll
      for (int h = 1; h >= 0; --h)
#pragma unroll
        for (int n = 0; n < NT; n += 2) {
          uint32_t b[4];
          const int r = kk * 16 + (lane & 15), c = h * (RP / 8) + n + (lane >> 4);
          ldsm4t(b, ls + r * L::kLPitch + c * 16);
          if constexpr (!BF16) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              __half2 v = __hmul2(*reinterpret_cast<__half2*>(&b[i]), (i & 1) ? f1 : f0);
              b[i] = *reinterpret_cast<uint32_t*>(&v);
            }
          }
#pragma unroll
          for (int m = 0; m < 2; ++m) {
            mma<BF16>(acc[m][n], a[m], b[0], b[1]);
            mma<BF16>(acc[m][n + 1], a[m], b[2], b[3]);
          }
        }
    }
  }
  cp_async_wait_group<0>();
  __syncthreads();

  float* red = reinterpret_cast<float*>(sm);  // [128 columns][RP]
  {
    const int g = lane >> 2, q = lane & 3;
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          red[(warp * 32 + m * 16 + g + (i >> 1) * 8) * L::kRedPitch + n * 8 + 2 * q + (i & 1)] = acc[m][n][i] * top;
  }
  if (cs > 1)
    cluster_sync();
  else
    __syncthreads();
  // two neighbours of the result per thread; the CTAs of the cluster share the columns
  const int cols = 128 / cs, cb = crank * cols;
  uint16_t* out = p.out + static_cast<int64_t>(adapter) * rank * p.len;
  for (int at = tid; at < cols * rank / 2; at += kThreads) {
    int c[2], r[2];
    if (p.rank_rows) {
      const int half = cols / 2;
      c[0] = cb + (at % half) * 2;
      c[1] = c[0] + 1;
      r[0] = r[1] = at / half;
    } else {
      const int half = rank / 2;
      c[0] = c[1] = cb + at / half;
      r[0] = (at % half) * 2;
      r[1] = r[0] + 1;
    }
    if (c0 + c[0] >= p.len) continue;
    float f[8][2], v[2] = {0.f, 0.f};
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k < cs)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint32_t a = smem_u32(red + c[i] * L::kRedPitch + r[i]);
          f[k][i] = ld_cluster_f32(cs > 1 ? mapa_shared(a, k) : a);
        }
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k < cs)
#pragma unroll
        for (int i = 0; i < 2; ++i) v[i] += f[k][i];
    const int64_t to = p.rank_rows ? static_cast<int64_t>(r[0]) * p.len + c0 + c[0]
                                   : static_cast<int64_t>(c0 + c[0]) * rank + r[0];
    *reinterpret_cast<uint32_t*>(out + to) = Half<BF16>::put2(v[0], v[1]);
  }
  if (cs > 1) cluster_sync();
}

template <bool BF16, int RT>
cudaError_t outer_as(const LoraRows& rows, const OuterParams (&p)[2], int rank, int sms, cudaStream_t s) {
  const int t0 = (p[0].len + 127) / 128, t1 = (p[1].len + 127) / 128;
  // shares of an adapter's rows: as many as fill the SMs four times over, each of 128 rows or more on average
  int cs = 1;
  while (cs < 8 && static_cast<int64_t>(t0 + t1) * rows.adapters * cs < 4 * sms &&
         rows.m / rows.adapters >= 256 * cs)
    cs *= 2;
  auto kernel = outer_kernel<BF16, RT>;
  const size_t smem = OuterSmem<RT>::kBytes;
  if (const cudaError_t e = allow_smem(kernel, smem); e != cudaSuccess) return e;
  return launch_pdl(kernel, dim3(static_cast<unsigned>((t0 + t1) * cs), static_cast<unsigned>(rows.adapters)),
                    dim3(kThreads), smem, cs, s, rows, p[0], p[1], rank, cs, t0);
}

}  // namespace

cudaError_t launch_lora_outer(const LoraRows& rows, const OuterParams (&p)[2], int rank, bool bf16, int sms,
                              cudaStream_t s) {
  return with_rank(rank, [&](auto rt) {
    constexpr int RT = decltype(rt)::value;
    return bf16 ? outer_as<true, RT>(rows, p, rank, sms, s) : outer_as<false, RT>(rows, p, rank, sms, s);
  });
}

}  // namespace wqmm
