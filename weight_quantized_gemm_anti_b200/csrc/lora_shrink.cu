// lora_shrink.cu -- the low-rank adapters' contractions over a long axis, low = scale * x W^T.
#include "lora_few.cuh"
#include "lora_tc.cuh"

namespace wqmm {
namespace {

// ------------------------------------------------------------------ the shares' sums
// A tile of BM rows is shared by the CTAs of a cluster, each with a part of the
// contraction.  CTA c finishes the BM / cs rows from c * BM / cs: the others write
// their sums of these into its shared memory, [CTA][row][PITCH], and it adds them
// in the order of the CTAs, so the result does not depend on timing.  Then scale,
// the row's power of two (float16) and the two 16-bit numbers.  Called by
// kThreads threads, tid 0 ...
template <int BM, int PITCH>
__device__ __forceinline__ uint32_t sums_of_row(const float* sums, int r, int cs, int crank) {
  const int own = BM / cs;
  const uint32_t at = smem_u32(sums + (crank * own + r % own) * PITCH);
  return cs > 1 ? mapa_shared(at, r / own) : at;
}

template <bool BF16, int RT, int BM, int PITCH>
__device__ __forceinline__ void finish_rows(const ShrinkParams& p, const Tile& tile, float scale, const float* sums,
                                            int cs, int crank, int tid) {
  constexpr int RP = RT * 16;
  constexpr int LANES = RP / 4, PER = kThreads / LANES;  // four values of a row per lane
  const int sub = tid % LANES, own = BM / cs;
  for (int r0 = 0; r0 < own; r0 += PER) {
    const int r = r0 + tid / LANES;
    const int place = tile.p0 + crank * own + r;
    const bool live = r < own && place < tile.p1;
    float v[4] = {0.f, 0.f, 0.f, 0.f};
    if (live) {
#pragma unroll
      for (int c = 0; c < 8; ++c)
        if (c < cs) {
          const float4 f = *reinterpret_cast<const float4*>(sums + (c * own + r) * PITCH + sub * 4);
          v[0] += f.x;
          v[1] += f.y;
          v[2] += f.z;
          v[3] += f.w;
        }
    }
    uint2 hi, lo;
    const float factor = split_row<BF16, LANES>(v, scale, hi, lo);
    if (live) {
      if (!BF16 && sub == 0) p.out.factor[place] = factor;
      uint16_t* o = p.out.low + static_cast<int64_t>(place) * (2 * RP) + sub * 4;
      *reinterpret_cast<uint2*>(o) = hi;
      *reinterpret_cast<uint2*>(o + RP) = lo;
    }
  }
}

// ------------------------------------------------------------------ few rows
// The gradients' two contractions in tiles of 16 rows: four warps split the
// contraction.  A chain of latencies bounds it: the order, the rows and weights,
// the cluster's exchange.

// Rank-major weights are staged in shared memory, 64 steps of the contraction at
// a time, so that the transposing load can make the instruction's operand of them.
template <int RT>
struct FewSmem {
  static constexpr int RP = RT * 16;
  static constexpr int kX = 16 * 128;
  static constexpr int kWPitch = RP * 2 + 16;
  static constexpr int kStage = kX + 64 * kWPitch;
  static constexpr int kStages = 4;
  static constexpr int kRed = 5 * 16 * RP * 4;  // the tile's sums, and the four warps' behind them
};

template <bool BF16, int RT>
__device__ __forceinline__ void few_rows_staged_sum(const LoraRows& rows, const ShrinkParams& p, int rank,
                                                    const Tile& tile, int s0, int s1, uint8_t* sm,
                                                    float (&acc)[RT * 2][4]) {
  constexpr int RP = RT * 16, NT = RT * 2;
  using L = FewSmem<RT>;
  constexpr int S = L::kStages;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t base = smem_u32(sm);
  const uint16_t* w = p.w + static_cast<int64_t>(tile.group) * rank * p.len;
  // this thread's part of x: 16-byte chunk tid % 8 of row tid / 8
  const int xc = tid & 7, xr = tid / 8;
  const int row = row_at(rows, tile.p0 + xr, tile.p1);
  const uint16_t* x = p.x.p + (row >= 0 ? row * p.x.ld : 0);
  auto load = [&](int step, int stage) {
    const uint32_t xs = base + stage * L::kStage, ws = xs + L::kX;
    const int k = step * 64 + xc * 8;
    const bool xhas = row >= 0 && k < p.len;
    cp16(xs + xr * 128 + ((xc ^ (xr & 7)) * 16), xhas ? x + k : p.x.p, xhas);
    constexpr int C = RP / 8;  // chunks of a row
#pragma unroll
    for (int i = 0; i < 64 * C / kThreads; ++i) {
      const int at = tid + i * kThreads, r = at / C, c = at % C, kk = step * 64 + r;
      const bool has = kk < p.len && c * 8 < rank;
      cp16(ws + r * L::kWPitch + c * 16, has ? w + static_cast<int64_t>(kk) * rank + c * 8 : w, has);
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
    uint32_t a[4];
    const int r = lane & 15, c = warp * 2 + (lane >> 4);
    ldsm4(a, xs + r * 128 + ((c ^ (r & 7)) * 16));
#pragma unroll
    for (int n = 0; n < NT; n += 2) {
      uint32_t b[4];
      ldsm4t(b, ws + (warp * 16 + (lane & 15)) * L::kWPitch + (n + (lane >> 4)) * 16);
      mma<BF16>(acc[n], a, b[0], b[1]);
      mma<BF16>(acc[n + 1], a, b[2], b[3]);
    }
  }
  cp_async_wait_group<0>();
  __syncthreads();
}

template <bool BF16, int RT, bool KM>
__device__ __forceinline__ void few_rows_tile(const LoraRows& rows, const ShrinkParams& p, int rank, int cs,
                                              const Tile& tile, uint8_t* sm) {
  constexpr int RP = RT * 16, NT = RT * 2;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int crank = cs > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int steps = (p.len + 63) / 64;
  const int s0 = static_cast<int>(static_cast<int64_t>(steps) * crank / cs);
  const int s1 = static_cast<int>(static_cast<int64_t>(steps) * (crank + 1) / cs);
  const float scale = p.scale ? p.scale[tile.group] : 1.f;
  float acc[NT][4];
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[n][i] = 0.f;
  if constexpr (KM)
    few_rows_sum<BF16, RT, 4>(rows, p, rank, tile, s0 * 64, min(s1 * 64, p.len), acc);
  else
    few_rows_staged_sum<BF16, RT>(rows, p, rank, tile, s0, s1, sm, acc);

  // the warps' sums, then the CTA's, then the cluster's
  float* sums = reinterpret_cast<float*>(sm + (KM ? 0 : FewSmem<RT>::kStage * FewSmem<RT>::kStages));
  float* part = sums + 16 * RP;
  {
    float* mine = part + warp * 16 * RP;
    const int g = lane >> 2, q = lane & 3;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      *reinterpret_cast<float2*>(mine + g * RP + n * 8 + 2 * q) = make_float2(acc[n][0], acc[n][1]);
      *reinterpret_cast<float2*>(mine + (g + 8) * RP + n * 8 + 2 * q) = make_float2(acc[n][2], acc[n][3]);
    }
  }
  __syncthreads();
  if (cs > 1) cluster_wait();  // the others have begun
  for (int at = tid * 4; at < 16 * RP; at += kThreads * 4) {
    const float4 v = sum_of_warps<4>(part + at, 16 * RP);
    st_cluster_f32x4(sums_of_row<16, RP>(sums, at / RP, cs, crank) + at % RP * 4, v.x, v.y, v.z, v.w);
  }
  if (cs > 1) {
    cluster_arrive();
    cluster_wait();
  } else {
    __syncthreads();
  }
  finish_rows<BF16, RT, 16, RP>(p, tile, scale, sums, cs, crank, tid);
}

template <bool BF16, int RT>
__global__ void __launch_bounds__(kThreads) shrink_few_kernel(LoraRows rows, ShrinkParams p0, ShrinkParams p1,
                                                              int rank, int cs) {
  extern __shared__ __align__(128) uint8_t sm[];
  pdl_wait();
  pdl_trigger();
  Tile tile;
  if (!find_tile(rows, 0, 16, blockIdx.x / cs, tile)) return;  // the same for the whole cluster
  if (cs > 1) cluster_arrive();
  if (blockIdx.y == 0)
    few_rows_tile<BF16, RT, true>(rows, p0, rank, cs, tile, sm);
  else
    few_rows_tile<BF16, RT, false>(rows, p1, rank, cs, tile, sm);
}

// ------------------------------------------------------------------ many rows
// Tiles of 128 rows on the tensor cores: D[128 rows][RP] += x[128][64] W[64][RP]
// in steps of 64 of the contraction.  Four warps copy x and W and read the sums
// at the end, one issues the MMAs.  A k-major W is K-major for the MMA, a
// rank-major one MN-major.  The copies of x bound the steps (about 800 cycles each,
// 22 bytes per clock and SM, the memory's rate); the start (2 us until the first
// stage is there) and the exchange and conversion at the end (2 us) come on top:
// both contractions of the gradients, 4096 rows of 4096, one adapter of rank 16,
// 67 MB: 17 us.
template <int RT>
struct ShrinkTc {
  static constexpr int RP = RT * 16;
  static constexpr int kX = 128 * 128, kW = RP * 128;
  static constexpr int kStage = kX + kW;
  static constexpr int kStages = RT == 1 ? 5 : RT == 2 ? 4 : RT == 4 ? 3 : 4;  // two CTAs per SM; one of rank 128
  static constexpr int kPerSm = RT == 8 ? 1 : 2;
  static constexpr int kPitch = RP + 4;  // of the sums, floats: rows a bank group apart
  static constexpr int kBytes = kStage * kStages + 128 * kPitch * 4 + 1024;
  static constexpr uint32_t kCols = RP < 32 ? 32 : RP;
};
constexpr int kShrinkThreads = kCopyThreads + 32;

template <bool BF16, int RT, bool KM>
__device__ __forceinline__ void shrink_copies(const ShrinkParams& p, int rank, const Tile& tile,
                                              const uint16_t* const (&x)[8], int s0, int n, uint32_t base,
                                              uint64_t* full, uint64_t* empty, volatile int* abort, uint32_t* err) {
  using L = ShrinkTc<RT>;
  constexpr int S = L::kStages;
  const int tid = threadIdx.x;
  const uint16_t* w = p.w + static_cast<int64_t>(tile.group) * rank * p.len;
  // 16-byte chunk c of rows tid / 8 + 16 i of x (and of a k-major W)
  const int c = tid & 7, r = tid >> 3;
  const uint32_t to = swizzled<128>(r, c);
  for (int i = 0; i < n; ++i) {
    const int st = i % S;
    if (i >= S && !warp_wait(&empty[st], ((i / S) & 1) ^ 1, abort, err, kDevTimeoutProducer)) break;
    const uint32_t xs = base + st * L::kStage, ws = xs + L::kX;
    const int k = (s0 + i) * 64 + c * 8;
    const bool in = k < p.len;
#pragma unroll
    for (int j = 0; j < 8; ++j) cp16(xs + to + j * 2048, in && x[j] ? x[j] + k : p.x.p, in && x[j]);
    if constexpr (KM) {
#pragma unroll
      for (int j = 0; j < RT; ++j) {
        const bool has = in && r + 16 * j < rank;
        cp16(ws + to + j * 2048, has ? w + static_cast<int64_t>(r + 16 * j) * p.len + k : w, has);
      }
    } else {
#pragma unroll
      for (int j = 0; j < RT; ++j) {
        const int at = tid + j * kCopyThreads, wr = at / (2 * RT), wc = at % (2 * RT), kk = (s0 + i) * 64 + wr;
        const bool has = kk < p.len && wc * 8 < rank;
        cp16(ws + RankRows<RT>::at(wr, wc), has ? w + static_cast<int64_t>(kk) * rank + wc * 8 : w, has);
      }
    }
    hand_over(&full[st]);
  }
  copies_landed();
}

template <bool BF16, int RT, bool BOTH>
__global__ void __launch_bounds__(kShrinkThreads) shrink_tc_kernel(LoraRows rows, ShrinkParams p0, ShrinkParams p1,
                                                                   int rank, int cs, uint32_t* err) {
  using L = ShrinkTc<RT>;
  using W = RankRows<RT>;
  constexpr int S = L::kStages, RP = L::RP;
  extern __shared__ uint8_t raw[];
  __shared__ __align__(8) uint64_t full[S], empty[S], done;
  __shared__ uint32_t tmem_sh;
  __shared__ int abort_sh;
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5;
  const bool km = !BOTH || blockIdx.y == 0;
  const ShrinkParams& p = km ? p0 : p1;
  if (threadIdx.x == 0) {
    for (int i = 0; i < S; ++i) {
      mbar_init(&full[i], 4);
      mbar_init(&empty[i], 1);
    }
    mbar_init(&done, 1);
    abort_sh = 0;
    fence_barrier_init();
  }
  pdl_wait();
  Tile tile;
  if (!find_tile(rows, 0, 128, blockIdx.x / cs, tile)) return;  // the same for the whole cluster
  if (cs > 1) cluster_arrive();
  if (warp == 4) {
    tmem_alloc(&tmem_sh, L::kCols);
    tmem_relinquish();
  }
  // rows tid / 8 + 16 i of the tile
  const uint16_t* x[8];
  if (warp < 4) {
    int v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = row_at(rows, tile.p0 + (threadIdx.x >> 3) + 16 * i, tile.p1);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = v[i] >= 0 ? p.x.p + v[i] * p.x.ld : nullptr;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_trigger();
  const uint32_t tmem = tmem_sh;
  volatile int* abort = &abort_sh;
  const int crank = cs > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int steps = (p.len + 63) / 64;
  const int s0 = static_cast<int>(static_cast<int64_t>(steps) * crank / cs);
  const int n = static_cast<int>(static_cast<int64_t>(steps) * (crank + 1) / cs) - s0;  // this CTA's steps
  const uint32_t base = smem_u32(sm);
  const float scale = p.scale ? p.scale[tile.group] : 1.f;

  if (warp < 4) {
    if (km)
      shrink_copies<BF16, RT, true>(p, rank, tile, x, s0, n, base, full, empty, abort, err);
    else
      shrink_copies<BF16, RT, false>(p, rank, tile, x, s0, n, base, full, empty, abort, err);
  } else {
    constexpr uint32_t kIdesc = idesc_make(1u, BF16 ? 1u : 0u, 128, RP);
    constexpr uint64_t kKBits = operand_bits(128, 16, 1024);
    for (int i = 0; i < n; ++i) {
      const int st = i % S;
      if (!stage_wait(&full[st], (i / S) & 1, abort, err)) break;
      const uint32_t xs = base + st * L::kStage, ws = xs + L::kX;
      if (elect_one()) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint64_t a = operand(xs + k * 32, kKBits);
          if (km)
            mma_f16_ss(tmem, a, operand(ws + k * 32, kKBits), kIdesc, i > 0 || k > 0);
          else
            mma_f16_ss(tmem, a, operand(ws + k * W::kStep, W::kBits), kIdesc | kBMn, i > 0 || k > 0);
        }
        mma_commit(&empty[st]);
      }
      __syncwarp();
    }
    if (elect_one()) mma_commit(&done);
    __syncwarp();
    volatile int no_abort = 0;
    warp_wait(&done, 0, &no_abort, err, kDevTimeoutDrain);
  }
  __syncthreads();  // the MMAs are done
  if (cs > 1) cluster_wait();  // the others have begun

  float* sums = reinterpret_cast<float*>(sm + L::kStage * S);
  if (warp < 4) {
    tc_fence_after();
    const uint32_t mine = sums_of_row<128, L::kPitch>(sums, threadIdx.x, cs, crank);  // warp w reads lanes 32 w ..
#pragma unroll
    for (int c = 0; c < RP; c += 16) {
      uint32_t v[16];
      if (n > 0) {
        tmem_ld_x16(tmem + (static_cast<uint32_t>(warp * 32) << 16) + c, v);
        tmem_wait_ld_r16(v);
      } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = 0;
      }
#pragma unroll
      for (int i = 0; i < 16; i += 4)
        st_cluster_f32x4(mine + (c + i) * 4, __uint_as_float(v[i]), __uint_as_float(v[i + 1]), __uint_as_float(v[i + 2]),
                         __uint_as_float(v[i + 3]));
    }
    tc_fence_before();
  }
  __syncthreads();
  if (cs > 1) {
    cluster_arrive();
    cluster_wait();
  }
  if (warp == 4) {
    tc_fence_after();
    tmem_dealloc(tmem, L::kCols);
  } else {
    finish_rows<BF16, RT, 128, L::kPitch>(p, tile, scale, sums, cs, crank, threadIdx.x);
  }
}

// ------------------------------------------------------------------ launches
// Shares of the contractions, at most 8: such that the longer one's shares are
// as long as an even deal of all steps of 64 to `room` CTAs makes them, or
// longer, and have at least four steps.
int shares(int64_t tiles, const ShrinkParams* p, int count, int64_t room) {
  int64_t all = 0, longest = 0;
  for (int i = 0; i < count; ++i) {
    const int64_t steps = (p[i].len + 63) / 64;
    all += tiles * steps;
    longest = std::max(longest, steps);
  }
  int cs = 1;
  while (cs < 8 && 2 * cs * all <= longest * room && longest >= 8 * cs) cs *= 2;
  return cs;
}

template <bool BF16, int RT>
cudaError_t shrink_few(const LoraRows& rows, const ShrinkParams* p, int rank, int sms, cudaStream_t s) {
  const int64_t tiles = most_tiles(rows.m, rows.adapters, 16);
  const int cs = shares(tiles, p, 2, 8 * sms);
  constexpr size_t smem = FewSmem<RT>::kRed + FewSmem<RT>::kStage * FewSmem<RT>::kStages;
  auto kernel = shrink_few_kernel<BF16, RT>;
  if (const cudaError_t e = allow_smem(kernel, smem); e != cudaSuccess) return e;
  return launch_pdl(kernel, dim3(static_cast<unsigned>(tiles * cs), 2), dim3(kThreads), smem, cs, s, rows, p[0], p[1],
                    rank, cs);
}

template <bool BF16, int RT, bool BOTH>
cudaError_t shrink_many(const LoraRows& rows, const ShrinkParams* p, int rank, int sms, cudaStream_t s) {
  const int64_t tiles = most_tiles(rows.m, rows.adapters, 128);
  // as many CTAs as run at once, but for SMs that a cluster's placement leaves free
  const int cs = shares(tiles, p, BOTH ? 2 : 1, ShrinkTc<RT>::kPerSm * sms * 7 / 8);
  auto kernel = shrink_tc_kernel<BF16, RT, BOTH>;
  if (const cudaError_t e = allow_smem(kernel, ShrinkTc<RT>::kBytes); e != cudaSuccess) return e;
  return launch_pdl(kernel, dim3(static_cast<unsigned>(tiles * cs), BOTH ? 2 : 1), dim3(kShrinkThreads),
                    ShrinkTc<RT>::kBytes, cs, s, rows, p[0], p[BOTH ? 1 : 0], rank, cs, device_error_word());
}

}  // namespace

int lora_padded_rank(int rank) { return 16 * padded_sixteenths(rank); }

bool lora_few_rows(const LoraRows& rows, int rank) { return few_rows(rows, rank); }

cudaError_t launch_lora_shrink(const LoraRows& rows, const ShrinkParams* p, int count, int rank, bool bf16, int sms,
                               cudaStream_t s) {
  return with_rank(rank, [&](auto rt) {
    constexpr int RT = decltype(rt)::value;
    auto by_count = [&](auto t) {
      constexpr bool T = decltype(t)::value;
      if (count == 1) {
        if constexpr (RT > 1) return shrink_many<T, RT, false>(rows, p, rank, sms, s);
        return cudaErrorInvalidValue;  // a forward pass at rank 16: lora_few.cu
      }
      return few_rows(rows, rank) ? shrink_few<T, RT>(rows, p, rank, sms, s)
                                  : shrink_many<T, RT, true>(rows, p, rank, sms, s);
    };
    return bf16 ? by_count(std::true_type()) : by_count(std::false_type());
  });
}

}  // namespace wqmm
