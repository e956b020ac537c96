// lora_outer.cu -- the gradients of the low-rank adapters' weights, contractions over the rows.
#include "lora_tc.cuh"

namespace wqmm {
namespace {

// D[128 columns of x][RP] += x[64 rows][128]^T low[64][RP] in steps of 64 rows
// of one adapter, on the tensor cores, both operands MN-major: a row of x and a
// row of low lie along the contraction as they are in memory.  low's two
// 16-bit numbers are two MMAs into the same sums.
//
// Roles: one warp gathers the rows of x (in the order of their adapters) and
// copies low's; one issues the MMAs; four write the sums; four put the
// operand low right where it is not as it was copied: rows behind the
// adapter's last belong to another one and become zeros (what they hold may
// not be finite), and float16 rows, whose powers of two differ, are brought to
// the largest of the CTA's rows.
//
// An item is 128 columns of one adapter's gradient.  With few items a cluster
// shares one, each CTA a part of the rows, and the parts meet in shared memory
// in the order of the CTAs; with many a CTA goes through several, the copies of
// the next under way while one is written (its sums are in tensor memory twice).
constexpr int kOuterThreads = 320;

template <int RT>
struct OuterTc {
  static constexpr int RP = RT * 16;
  static constexpr int kX = 2 * 64 * 128;             // two blocks of 64 columns
  static constexpr int kLow = RankRows<RT>::kBytes;   // one of the two numbers
  static constexpr int kStage = kX + 2 * kLow;
  static constexpr int kStages = RT == 1 ? 5 : RT == 2 ? 4 : RT == 4 ? 3 : 4;  // two CTAs per SM; one of rank 128
  static constexpr int kPerSm = RT == 8 ? 1 : 2;
  static constexpr int kBytes = kStage * kStages + 1024;
  static constexpr uint32_t kCols = 2 * RP < 32 ? 32 : 2 * RP;
  static constexpr int kPitch = RP + 1;  // of the sums, floats
  static_assert(128 * kPitch * 4 <= kStage * kStages, "the sums reuse the stages");
};

struct OuterMaps {
  CUtensorMap x[2];    // gathered rows: box 64 columns x 1 row, 128-byte swizzle
  CUtensorMap low[2];  // box 64 rows
};

// Two neighbours of the gradient: columns c (and c + 1 in the rank-row form), rank rows r (and r + 1 otherwise).
template <bool BF16>
__device__ __forceinline__ void put_pair(uint16_t* out, const OuterParams& p, int rank, int c, int r, float a, float b) {
  const int64_t to = p.rank_rows ? static_cast<int64_t>(r) * p.len + c : static_cast<int64_t>(c) * rank + r;
  *reinterpret_cast<uint32_t*>(out + to) = Half<BF16>::put2(a, b);
}

template <bool BF16, int RT>
__global__ void __launch_bounds__(kOuterThreads) outer_tc_kernel(LoraRows rows, OuterParams p0, OuterParams p1,
                                                                 const __grid_constant__ OuterMaps maps, int rank,
                                                                 int cs, int tiles0, int tiles, int items,
                                                                 uint32_t* err) {
  using L = OuterTc<RT>;
  using R = RankRows<RT>;
  constexpr int S = L::kStages, RP = L::RP;
  extern __shared__ uint8_t raw[];
  __shared__ __align__(8) uint64_t full[S], right[S], empty[S], sums_full[2], sums_empty[2], top_ready[2], done;
  __shared__ uint32_t tmem_sh;
  __shared__ int abort_sh;
  __shared__ float top_sh[2], tops[4];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  const uint32_t base = smem_u32(sm);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int crank = cs > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int first = blockIdx.x / cs, stride = gridDim.x / cs;

  if (threadIdx.x == 0) {
    for (int i = 0; i < S; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
      mbar_init(&right[i], 4);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sums_full[i], 1);
      mbar_init(&sums_empty[i], 128);
      mbar_init(&top_ready[i], 1);
    }
    mbar_init(&done, 1);
    abort_sh = 0;
    fence_barrier_init();
  }
  __syncthreads();
  volatile int* abort = &abort_sh;

  // an item's adapter, columns and steps; its rows are [r0, r1) in steps of 64 from r0 + 64 s0
  struct Item {
    int which, c0, adapter;
    int64_t r0, r1, s0;
    int n;
  };
  auto item_at = [&](int it) {
    Item o;
    o.adapter = it / tiles;
    const int ct = it % tiles;
    o.which = ct < tiles0 ? 0 : 1;
    o.c0 = (ct < tiles0 ? ct : ct - tiles0) * 128;
    o.r0 = offset_at(rows, o.adapter);
    o.r1 = max(offset_at(rows, o.adapter + 1), o.r0);
    const int64_t steps = (o.r1 - o.r0 + 63) / 64;
    o.s0 = steps * crank / cs;
    o.n = static_cast<int>(steps * (crank + 1) / cs - o.s0);
    return o;
  };
  // The copy warp's part: four rows of x per lane and step, and low's rows.
  const int quad4 = 4 * (lane & 15);
  int64_t next[4];
  auto find = [&](const Item& o, int i) {
#pragma unroll
    for (int j = 0; j < 4; ++j) next[j] = i < o.n ? row_at(rows, o.r0 + (o.s0 + i) * 64 + quad4 + j, o.r1) : -1;
  };
  auto copy_x = [&](const Item& o, int st) {
    int4 four;  // the row behind the last reads as zeros
    four.x = static_cast<int>(next[0] >= 0 ? next[0] : rows.m);
    four.y = static_cast<int>(next[1] >= 0 ? next[1] : rows.m);
    four.z = static_cast<int>(next[2] >= 0 ? next[2] : rows.m);
    four.w = static_cast<int>(next[3] >= 0 ? next[3] : rows.m);
    if (lane == 0) mbar_arrive_expect_tx(&full[st], L::kStage);
    __syncwarp();
    tma_gather4(base + st * L::kStage + (lane >> 4) * 8192 + (lane & 15) * 512, &maps.x[o.which], &full[st],
                o.c0 + (lane >> 4) * 64, four);
    __syncwarp();
  };
  auto copy_low = [&](const Item& o, int i, int st) {
    if (lane == 0) {
      const int r = static_cast<int>(o.r0 + (o.s0 + i) * 64);
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int b = 0; b < R::kBlocks; ++b)
          tma_load_2d(sm + st * L::kStage + L::kX + h * L::kLow + b * R::kBlock, &maps.low[o.which], &full[st],
                      h * RP + b * R::kCols, r);
    }
    __syncwarp();
  };
  // x and the order are older than the launch before this one, which has waited for all that came
  // before it: the first stages' rows of x are read while it ends, low after that
  int early = 0;
  if (warp == 0 && first < items) {
    const Item o = item_at(first);
    for (; early < S && early < o.n; ++early) {
      find(o, early);
      copy_x(o, early);
    }
  }
  pdl_wait();
  pdl_trigger();
  // tensor memory is taken now: the launch before this one may have held it all
  if (warp == 1) {
    tmem_alloc(&tmem_sh, L::kCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_sh;

  if (warp == 0) {
    int g = 0;
    bool live = true;
    for (int it = first; it < items && live; it += stride) {
      const Item o = item_at(it);
      const int had = it == first ? early : 0;
      for (int i = 0; i < had; ++i, ++g) copy_low(o, i, g % S);
      find(o, had);
      for (int i = had; i < o.n; ++i, ++g) {
        const int st = g % S;
        if (g >= S && !warp_wait(&empty[st], ((g / S) & 1) ^ 1, abort, err, kDevTimeoutProducer)) {
          live = false;
          break;
        }
        copy_x(o, st);
        copy_low(o, i, st);
        find(o, i + 1);
      }
    }
    if (lane == 0)  // every copy issued lands before the CTA may end
      for (int j = g > S ? g - S : 0; j < g; ++j) {
        volatile int no_abort = 0;
        mbar_wait(&full[j % S], (j / S) & 1, &no_abort, err, kDevTimeoutDrain);
      }
    __syncwarp();
  } else if (warp == 1) {
    constexpr uint32_t kIdesc = idesc_make(1u, BF16 ? 1u : 0u, 128, RP) | kAMn | kBMn;
    constexpr uint64_t kXBits = operand_bits(128, 8192, 1024);
    int g = 0, k = 0;
    bool live = true;
    for (int it = first; it < items && live; it += stride, ++k) {
      const Item o = item_at(it);
      const int buf = k & 1;
      if (k >= 2 && !warp_wait(&sums_empty[buf], ((k / 2) & 1) ^ 1, abort, err, kDevTimeoutMma)) break;
      tc_fence_after();
      const uint32_t d = tmem + buf * RP;
      for (int i = 0; i < o.n; ++i, ++g) {
        const int st = g % S;
        if (!warp_wait(&full[st], (g / S) & 1, abort, err, kDevTimeoutMma) ||
            !warp_wait(&right[st], (g / S) & 1, abort, err, kDevTimeoutMma)) {
          live = false;
          break;
        }
        tc_fence_after();
        const uint32_t xs = base + st * L::kStage, ls = xs + L::kX;
        if (elect_one()) {
#pragma unroll
          for (int h = 1; h >= 0; --h)  // the small part first
#pragma unroll
            for (int s = 0; s < 4; ++s)
              mma_f16_ss(d, operand(xs + s * 2048, kXBits), operand(ls + h * L::kLow + s * R::kStep, R::kBits), kIdesc,
                         i > 0 || h < 1 || s > 0);
          mma_commit(&empty[st]);
        }
        __syncwarp();
      }
      if (!live) break;
      if (elect_one()) mma_commit(&sums_full[buf]);
      __syncwarp();
    }
    if (elect_one()) mma_commit(&done);
    __syncwarp();
    volatile int no_abort = 0;
    warp_wait(&done, 0, &no_abort, err, kDevTimeoutDrain);
  } else if (warp >= 6) {
    // ---------------------------------------------------------------- low put right
    // (after a wait that gave up these warps still go through the loop, for the barriers among them)
    const int tid = threadIdx.x - 192;
    int g = 0, k = 0;
    bool live = true;
    for (int it = first; it < items; it += stride, ++k) {
      const Item o = item_at(it);
      const LoraLow& low = o.which == 0 ? p0.low : p1.low;
      const int64_t begin = o.r0 + o.s0 * 64;
      const int n = static_cast<int>(min(static_cast<int64_t>(o.n) * 64, o.r1 - begin));  // rows
      float below = 1.f;
      if constexpr (!BF16) {
        float top = 0.f;
        for (int r = tid; r < n; r += 128) top = fmaxf(top, low.factor[begin + r]);
#pragma unroll
        for (int s = 16; s > 0; s >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, s));
        named_bar_sync(1, 128);  // the last item's maxima are read
        if (lane == 0) tops[warp - 6] = top;
        named_bar_sync(1, 128);
        top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]));
        if (!(top > 0.f)) top = 1.f;  // no rows
        below = 1.f / top;            // of a power of two: exact
        // the maximum of two items ago has been read when its sums have
        live = live && (k < 2 || warp_wait(&sums_empty[k & 1], ((k / 2) & 1) ^ 1, abort, err, kDevTimeoutDequant));
        if (live && tid == 0) {
          top_sh[k & 1] = top;
          mbar_arrive(&top_ready[k & 1]);
        }
      }
      for (int i = 0; i < o.n; ++i, ++g) {
        const int st = g % S;
        constexpr int kChunks = 2 * L::kLow / 16 / 128;  // 16-byte chunks per thread
        float f[kChunks];
        if constexpr (!BF16) {
#pragma unroll
          for (int c = 0; c < kChunks; ++c) {
            const int r = i * 64 + (((tid + c * 128) * 16) % R::kBlock) / R::kRow;
            f[c] = r < n ? low.factor[begin + r] * below : 0.f;
          }
        }
        live = live && warp_wait(&full[st], (g / S) & 1, abort, err, kDevTimeoutDequant);
        if (!live) continue;
        if (!BF16 || (i + 1) * 64 > n) {
#pragma unroll
          for (int c = 0; c < kChunks; ++c) {
            const int r = i * 64 + (((tid + c * 128) * 16) % R::kBlock) / R::kRow;
            uint4* at = reinterpret_cast<uint4*>(sm + st * L::kStage + L::kX + (tid + c * 128) * 16);
            if (r >= n) {
              *at = make_uint4(0, 0, 0, 0);
            } else if constexpr (!BF16) {
              const __half2 by = __float2half2_rn(f[c]);
              const uint4 v = *at;
              uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const __half2 x = __hmul2(*reinterpret_cast<__half2*>(&w[j]), by);
                w[j] = *reinterpret_cast<const uint32_t*>(&x);
              }
              *at = make_uint4(w[0], w[1], w[2], w[3]);
            }
          }
          fence_proxy_async_smem();  // the MMA reads what was written here
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&right[st]);
      }
    }
  } else if (warp >= 2) {
    // ---------------------------------------------------------------- the sums
    const int quad = warp & 3;  // the lanes of tensor memory that this warp may read
    const int col = quad * 32 + lane;
    int k = 0;
    for (int it = first; it < items; it += stride, ++k) {
      const Item o = item_at(it);
      const OuterParams& p = o.which == 0 ? p0 : p1;
      const int buf = k & 1;
      if (!warp_wait(&sums_full[buf], (k / 2) & 1, abort, err, kDevTimeoutEpilogue)) break;
      float top = 1.f;
      if constexpr (!BF16) {
        if (!warp_wait(&top_ready[buf], (k / 2) & 1, abort, err, kDevTimeoutEpilogue)) break;
        top = top_sh[buf];
      }
      tc_fence_after();
      uint16_t* out = p.out + static_cast<int64_t>(o.adapter) * rank * p.len;
      float* red = reinterpret_cast<float*>(sm) + col * L::kPitch;  // a cluster's only item: the stages are free
#pragma unroll
      for (int c = 0; c < RP; c += 16) {
        uint32_t v[16];
        if (o.n > 0) {
          tmem_ld_x16(tmem + (static_cast<uint32_t>(quad * 32) << 16) + buf * RP + c, v);
          tmem_wait_ld_r16(v);
        } else {
#pragma unroll
          for (int i = 0; i < 16; ++i) v[i] = 0;
        }
        if (cs > 1) {
#pragma unroll
          for (int i = 0; i < 16; ++i) red[c + i] = __uint_as_float(v[i]) * top;
        } else if (p.rank_rows) {
          // a rank row's neighbours are in the neighbour lanes: pairs of two rows at a time
#pragma unroll
          for (int i = 0; i < 16; i += 2) {
            const float a = __uint_as_float(v[i]) * top, b = __uint_as_float(v[i + 1]) * top;
            const float other = __shfl_xor_sync(0xffffffffu, (lane & 1) ? a : b, 1);
            const int r = c + i + (lane & 1), cc = o.c0 + (col & ~1);
            if (r < rank && cc < p.len)
              put_pair<BF16>(out, p, rank, cc, r, (lane & 1) ? other : a, (lane & 1) ? b : other);
          }
        } else if (o.c0 + col < p.len) {
#pragma unroll
          for (int i = 0; i < 16; i += 8)
            if (c + i < rank) {
              uint4 w;
              w.x = Half<BF16>::put2(__uint_as_float(v[i]) * top, __uint_as_float(v[i + 1]) * top);
              w.y = Half<BF16>::put2(__uint_as_float(v[i + 2]) * top, __uint_as_float(v[i + 3]) * top);
              w.z = Half<BF16>::put2(__uint_as_float(v[i + 4]) * top, __uint_as_float(v[i + 5]) * top);
              w.w = Half<BF16>::put2(__uint_as_float(v[i + 6]) * top, __uint_as_float(v[i + 7]) * top);
              *reinterpret_cast<uint4*>(out + static_cast<int64_t>(o.c0 + col) * rank + c + i) = w;
            }
        }
      }
      tc_fence_before();
      mbar_arrive(&sums_empty[buf]);
    }
  }
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, L::kCols);
  }
  if (cs > 1) {
    cluster_sync();
    const Item o = item_at(first);
    const OuterParams& p = o.which == 0 ? p0 : p1;
    uint16_t* out = p.out + static_cast<int64_t>(o.adapter) * rank * p.len;
    const float* red = reinterpret_cast<const float*>(sm);
    // two neighbours of the result per thread; the CTAs of the cluster share the columns
    const int cols = 128 / cs, cb = crank * cols;
    for (int at = threadIdx.x; at < cols * rank / 2; at += kOuterThreads) {
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
      if (o.c0 + c[0] >= p.len) continue;
      float f[8][2], v[2] = {0.f, 0.f};
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j < cs)
#pragma unroll
          for (int i = 0; i < 2; ++i)
            f[j][i] = ld_cluster_f32(mapa_shared(smem_u32(red + c[i] * L::kPitch + r[i]), j));
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j < cs)
#pragma unroll
          for (int i = 0; i < 2; ++i) v[i] += f[j][i];
      put_pair<BF16>(out, p, rank, o.c0 + c[0], r[0], v[0], v[1]);
    }
    __syncwarp();
    cluster_sync();  // no CTA ends while another reads its sums
  }
}

// ------------------------------------------------------------------ launches
template <bool BF16, int RT>
cudaError_t outer_as(const LoraRows& rows, const OuterParams (&p)[2], const OuterMaps& maps, int rank, int sms,
                     cudaStream_t s) {
  using L = OuterTc<RT>;
  const int t0 = (p[0].len + 127) / 128, tiles = t0 + (p[1].len + 127) / 128;
  const int items = tiles * rows.adapters;
  const int room = L::kPerSm * sms;
  // shares of an adapter's rows: as many as there is room for at once, each of 128 rows or more on average
  int cs = 1;
  while (cs < 8 && static_cast<int64_t>(items) * cs * 2 <= room && rows.m / rows.adapters >= 256 * cs) cs *= 2;
  const int grid = cs > 1 ? items * cs : std::min(items, room);
  auto kernel = outer_tc_kernel<BF16, RT>;
  if (const cudaError_t e = allow_smem(kernel, L::kBytes); e != cudaSuccess) return e;
  return launch_pdl(kernel, dim3(static_cast<unsigned>(grid)), dim3(kOuterThreads), L::kBytes, cs, s, rows, p[0], p[1],
                    maps, rank, cs, t0, tiles, items, device_error_word());
}

}  // namespace

wqmm_status launch_lora_outer(const LoraRows& rows, const OuterParams (&p)[2], int rank, bool bf16, int sms,
                              cudaStream_t s) {
  OuterMaps maps;
  const int rp = lora_padded_rank(rank);
  for (int i = 0; i < 2; ++i) {
    const uint64_t m = static_cast<uint64_t>(rows.m);
    const uint64_t xe[2] = {static_cast<uint64_t>(p[i].len), m}, xs[1] = {static_cast<uint64_t>(p[i].x.ld) * 2};
    const uint32_t xb[2] = {64, 1};
    wqmm_status st = tensor_map16(&maps.x[i], p[i].x.p, bf16, 2, xe, xs, xb, 128);
    if (st) return st;
    const uint64_t le[2] = {static_cast<uint64_t>(2 * rp), m}, ls[1] = {static_cast<uint64_t>(4 * rp)};
    const uint32_t lb[2] = {static_cast<uint32_t>(std::min(rp, 64)), 64};
    st = tensor_map16(&maps.low[i], p[i].low.low, bf16, 2, le, ls, lb, static_cast<int>(lb[0]) * 2);
    if (st) return st;
  }
  const cudaError_t e = with_rank(rank, [&](auto rt) {
    constexpr int RT = decltype(rt)::value;
    return bf16 ? outer_as<true, RT>(rows, p, maps, rank, sms, s) : outer_as<false, RT>(rows, p, maps, rank, sms, s);
  });
  return e == cudaSuccess ? WQMM_SUCCESS : cuda_fail(e, "adapter weight gradient launch");
}

}  // namespace wqmm
