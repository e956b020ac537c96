// lora_few.cu -- the low-rank adapters' part at rank 16 or for few rows, both contractions in one launch.
#include "lora_few.cuh"

namespace wqmm {
namespace {

constexpr int kFewWarps = 8;
// CTAs per SM.  Told to the compiler too: up to rank 32 it then schedules for the registers of two, 23.4 us
// instead of 25.8 for 4096 rows of 4096 at rank 16.
template <int RT>
constexpr int kFewPerSm = RT < 4 ? 2 : 1;

// A cluster has a tile of 16 rows.  Its CTAs share the contraction over k, send
// each other their sums, finish the tile's low values (each CTA all of them, the
// parts added in the order of the CTAs) and share the columns of the result.
// No operand passes through shared memory but low.  The weights of
// the columns are read as those of the contraction are: 16 neighbouring bytes of
// a column's rank per thread, in the order that lets a thread add and store
// 16 bytes of a row at once (column q * 8 + 2 j + e of a group of 32 is column
// 2 q + e of the instruction's tile j).  The first columns' weights and y are
// under way while the sums are exchanged.
//
// Latencies bound few rows: the launch, the order, two rounds of loads, one
// exchange (k = n = 4096, rank 16: 1 row 4.9 us, 64 rows of four adapters 5.2);
// many, memory and the reads of the weights, again for each 16 rows (4096 rows:
// 22 us, 4.5 TB/s of x, y and the result).  One launch and no workspace also
// spare the host a launch and an allocation (8.2 us a call with them, 5.9 without).
template <int RT>
struct FewTile {
  static constexpr int RP = RT * 16;
  static constexpr int kLowPitch = 2 * RP + 8;  // 16-bit numbers: rows a bank group apart
  static constexpr int kSums = 8 * 16 * RP * 4, kPart = kFewWarps * 16 * RP * 4, kLow = 16 * kLowPitch * 2;
  static constexpr int kBytes = kSums + kPart + kLow + 64;
  static constexpr int kGroups = RT == 1 ? 2 : 1;      // of 32 columns, in flight per warp
  static constexpr int kLoads = RT == 1 ? 1 : RT / 2;  // of a column's rank
};

template <bool BF16, int RT>
__global__ void __launch_bounds__(kFewWarps * 32, kFewPerSm<RT>)
    few_kernel(LoraRows rows, ShrinkParams sp, ExpandParams p, int rank,
                                                             int cs) {
  using L = FewTile<RT>;
  constexpr int NW = kFewWarps, RP = L::RP, NT = RT * 2, U = L::kGroups, KL = L::kLoads;
  extern __shared__ __align__(128) uint8_t sm[];
  float* sums = reinterpret_cast<float*>(sm);  // [CTA][16][RP]
  float* part = reinterpret_cast<float*>(sm + L::kSums);
  uint16_t* low = reinterpret_cast<uint16_t*>(sm + L::kSums + L::kPart);
  float* factors = reinterpret_cast<float*>(sm + L::kSums + L::kPart + L::kLow);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, q = lane & 3;
  pdl_wait();
  pdl_trigger();
  Tile tile;
  if (!find_tile(rows, p.bare, 16, blockIdx.x / cs, tile)) return;  // the same for the whole cluster
  const bool with = tile.group < rows.adapters;
  const int crank = cs > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  if (with && cs > 1) cluster_arrive();

  // this thread's two rows of y and out, and its warp's groups of columns
  int row[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) row[i] = row_at(rows, tile.p0 + g + 8 * i, tile.p1);
  const int all = p.len / 32;
  const int g_end = static_cast<int>(static_cast<int64_t>(all) * (crank + 1) / cs);
  int grp = static_cast<int>(static_cast<int64_t>(all) * crank / cs) + warp;
  const uint16_t* w = p.w + (static_cast<int64_t>(with ? tile.group : 0) * p.len + (g >> 1) * 8 + (g & 1)) * rank;
  uint4 wv[U][4][KL], y[U][2], wn[U][4][KL], yn[U][2];
  auto fetch = [&](int grp) {
    const uint4 zero = make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int at = grp + u * NW;
      const bool in = at < g_end;
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int k = 0; k < KL; ++k) {
          const int r = RT == 1 ? q * 4 : k * 32 + q * 8;
          const uint16_t* from = w + (static_cast<int64_t>(at) * 32 + 2 * j) * rank + r;
          wn[u][j][k] = zero;
          if (with && in && r < rank) {
            if constexpr (RT == 1) {
              const uint2 v = *reinterpret_cast<const uint2*>(from);
              wn[u][j][k] = make_uint4(v.x, v.y, 0, 0);
            } else {
              wn[u][j][k] = *reinterpret_cast<const uint4*>(from);
            }
          }
        }
#pragma unroll
      for (int i = 0; i < 2; ++i)
        yn[u][i] = in && p.y.p && row[i] >= 0
                       ? *reinterpret_cast<const uint4*>(p.y.p + row[i] * p.y.ld + at * 32 + q * 8)
                       : zero;
    }
  };

  uint32_t a[2][RT][4];  // hi, lo
  float factor[2] = {1.f, 1.f};
  if (with) {
    const float scale = sp.scale ? sp.scale[tile.group] : 1.f;
    const int steps = sp.len / 32;
    const int k0 = static_cast<int>(static_cast<int64_t>(steps) * crank / cs) * 32;
    const int k1 = static_cast<int>(static_cast<int64_t>(steps) * (crank + 1) / cs) * 32;
    float acc[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[n][i] = 0.f;
    few_rows_sum<BF16, RT, NW>(rows, sp, rank, tile, k0, k1, acc);
    fetch(grp);
    float* mine = part + warp * 16 * RP;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      *reinterpret_cast<float2*>(mine + g * RP + n * 8 + 2 * q) = make_float2(acc[n][0], acc[n][1]);
      *reinterpret_cast<float2*>(mine + (g + 8) * RP + n * 8 + 2 * q) = make_float2(acc[n][2], acc[n][3]);
    }
    __syncthreads();
    if (cs > 1) cluster_wait();  // the others have begun
    for (int at = tid * 4; at < 16 * RP; at += NW * 32 * 4) {
      const float4 v = sum_of_warps<NW>(part + at, 16 * RP);
      const uint32_t to = smem_u32(sums + crank * 16 * RP + at);
      for (int c = 0; c < cs; ++c) st_cluster_f32x4(cs > 1 ? mapa_shared(to, c) : to, v.x, v.y, v.z, v.w);
    }
    if (cs > 1) {
      cluster_arrive();
      cluster_wait();
    } else {
      __syncthreads();
    }
    constexpr int LANES = RP / 4, PER = NW * 32 / LANES;
    for (int r0 = 0; r0 < 16; r0 += PER) {
      const int r = r0 + tid / LANES, sub = tid % LANES;
      float v[4] = {0.f, 0.f, 0.f, 0.f};
      if (r < 16) {
#pragma unroll
        for (int c = 0; c < 8; ++c)
          if (c < cs) {
            const float4 f = *reinterpret_cast<const float4*>(sums + (c * 16 + r) * RP + sub * 4);
            v[0] += f.x;
            v[1] += f.y;
            v[2] += f.z;
            v[3] += f.w;
          }
      }
      uint2 hi, lo;
      const float f = split_row<BF16, LANES>(v, scale, hi, lo);
      if (r < 16) {
        *reinterpret_cast<uint2*>(low + r * L::kLowPitch + sub * 4) = hi;
        *reinterpret_cast<uint2*>(low + r * L::kLowPitch + RP + sub * 4) = lo;
        if (sub == 0) factors[r] = f;
      }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t* from = reinterpret_cast<const uint32_t*>(low + (g + 8 * i) * L::kLowPitch);
      if constexpr (!BF16) factor[i] = factors[g + 8 * i];
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int k = 0; k < RT; ++k) {
          // the words that stand beside the weights' of the same load
          const int at = h * (RP / 2) + (RT == 1 ? q * 2 : k / 2 * 16 + q * 4 + k % 2 * 2);
          a[h][k][i] = from[at];
          a[h][k][i + 2] = from[at + 1];
        }
    }
  } else {
    fetch(grp);
  }

  for (; grp < g_end; grp += U * NW) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int k = 0; k < KL; ++k) wv[u][j][k] = wn[u][j][k];
      y[u][0] = yn[u][0];
      y[u][1] = yn[u][1];
    }
    fetch(grp + U * NW);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int col = (grp + u * NW) * 32 + q * 8;
      float acc[4][4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[j][i] = 0.f;
      if (with) {
#pragma unroll
        for (int k = 0; k < RT; ++k)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint4 v = wv[u][j][RT == 1 ? 0 : k / 2];
            const uint32_t b0 = k % 2 ? v.z : v.x, b1 = k % 2 ? v.w : v.y;
            mma<BF16>(acc[j], a[1][k], b0, b1);  // the small part first
            mma<BF16>(acc[j], a[0][k], b0, b1);
          }
      }
      if (grp + u * NW >= g_end) continue;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if (row[i] < 0) continue;
        const uint32_t yv[4] = {y[u][i].x, y[u][i].y, y[u][i].z, y[u][i].w};
        uint32_t o[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float v0 = acc[j][2 * i], v1 = acc[j][2 * i + 1];
          const float y0 = Half<BF16>::get(yv[j] & 0xffff), y1 = Half<BF16>::get(yv[j] >> 16);
          v0 = BF16 ? v0 + y0 : fmaf(factor[i], v0, y0);
          v1 = BF16 ? v1 + y1 : fmaf(factor[i], v1, y1);
          o[j] = with ? Half<BF16>::put2(v0, v1) : yv[j];
        }
        *reinterpret_cast<uint4*>(p.out + row[i] * p.ldo + col) = make_uint4(o[0], o[1], o[2], o[3]);
      }
    }
  }
}

// Places for CTAs at once: seven eighths of the SMs' (two or one each, by the registers), since a cluster's stay
// within one group of SMs (rank 64, 256 rows: 136 in clusters of eight 15.8 us, 68 in clusters of four 10.6).
template <int RT>
int few_places(int sms) {
  return kFewPerSm<RT> * sms * 7 / 8;
}

template <bool BF16, int RT>
cudaError_t few_as(const LoraRows& rows, const ShrinkParams& sp, const ExpandParams& ep, int rank, int sms,
                   cudaStream_t s) {
  auto kernel = few_kernel<BF16, RT>;
  constexpr size_t smem = FewTile<RT>::kBytes;
  if (const cudaError_t e = allow_smem(kernel, smem); e != cudaSuccess) return e;
  // CTAs of a tile: as many as find room at once
  const int64_t tiles = most_tiles(rows.m, rows.adapters + ep.bare, 16);
  int cs = 1;
  while (cs < 8 && tiles * cs * 2 <= few_places<RT>(sms)) cs *= 2;
  return launch_pdl(kernel, dim3(static_cast<unsigned>(tiles * cs)), dim3(kFewWarps * 32), smem, cs, s, rows, sp, ep,
                    rank, cs);
}

}  // namespace

// The one launch reads an adapter's weights again for each 16 of its rows, the two
// of lora_shrink.cu and lora_expand.cu for each 128.  At rank 16 that costs less
// than the second launch at any length; above, the rows up to which it is ahead
// fall with the rank: 4096 at rank 32; at rank 64 as many as make clusters of two
// CTAs per tile, whose shares of the contraction halve its length, and of four
// at rank 128.  Few rows per adapter leave it ahead.  k = n = 4096 (4096 x 1024
// is more in its favour, 1024 x 8192 less), one launch and two, in us:
//   one adapter   rank 16  1000 rows 8.5, 11.9   4096 rows 22.2, 29.4  16384 rows 86.8, 95.8
//                 rank 32  1000 rows 10.3, 14.0  4096 rows 30.4, 32.6   8192 rows 60.5, 56.5
//                 rank 64   400 rows 10.4, 15.2  1000 rows 15.7, 16.6   1024 rows 20.7, 16.6
//                 rank 128  150 rows 12.5, 16.7   400 rows 15.5, 18.9    512 rows 21.9, 19.1
//   24 adapters   rank 16  1000 rows 11.5, 15.6  4096 rows 23.7, 32.3  16384 rows 87.8, 99.5
//                 rank 32  2048 rows 22.1, 24.1  4096 rows 32.8, 36.8   8192 rows 62.9, 58.7
//                 rank 64   512 rows 14.9, 24.5  1000 rows 25.1, 25.4   2000 rows 31.5, 29.5
//                 rank 128  256 rows 23.7, 30.4   512 rows 25.5, 31.6   1000 rows 47.8, 33.2
//   64 adapters   rank 64  1024 rows 34.2, 44.2  2000 rows 70.1, 47.7
//                 rank 128  512 rows 55.9, 72.4  1000 rows 57.4, 73.5
bool lora_one_launch(const LoraRows& r, int rank, int bare, int sms) {
  if (rank <= 16 || r.m <= 16 * static_cast<int64_t>(r.adapters)) return true;
  if (rank <= 32) return r.m <= 4096;
  return most_tiles(r.m, r.adapters + bare, 16) * (rank <= 64 ? 2 : 4) <= few_places<4>(sms);
}

cudaError_t launch_lora_few(const LoraRows& rows, const ShrinkParams& sp, const ExpandParams& ep, int rank, bool bf16,
                            int sms, cudaStream_t s) {
  return with_rank(rank, [&](auto rt) {
    constexpr int RT = decltype(rt)::value;
    return bf16 ? few_as<true, RT>(rows, sp, ep, rank, sms, s) : few_as<false, RT>(rows, sp, ep, rank, sms, s);
  });
}

}  // namespace wqmm
