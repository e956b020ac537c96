// lora_outer.cu -- the gradients of the low-rank adapters' weights, contractions over the rows.
#include "lora_tc.cuh"

namespace wqmm {
namespace {

// D[128 columns of x][RP] += x[64 rows][128]^T low[64][RP] in steps of 64 rows
// of one adapter, on the tensor cores, both operands MN-major: a row of x and a
// row of low lie along the contraction as they are in memory.  low's two
// 16-bit numbers are two MMAs into the same sums.
//
// Roles: four warps copy the rows of x (in the order of their adapters), four
// those of low, one issues the MMAs, four write the sums.  Rows behind the adapter's last
// are zeros in both operands.  float16 rows of low have a power of two each;
// on their way to shared memory they are brought to the largest of the CTA's rows,
// where a value's two numbers are off by 2^-25 each: 2^-38 of the largest value.
//
// An item is 128 columns of one adapter's gradient.  With few items a cluster
// shares one, each CTA a part of the rows, and the parts meet in shared memory
// in the order of the CTAs; with many a CTA goes through several, the copies of
// the next under way while one is written (its sums are in tensor memory twice).
//
// The copies bound it.  One adapter of rank 16, 4096 rows of x and of the gradient,
// 4096 each, 67 MB: 17 us behind the contractions that read the same (24 us from
// memory alone); six adapters of rank 64, float16, 2051 rows of 8192 and 1024: 28 us,
// where a step's low rows are as many bytes as its x and pass through registers.
// With the copies issued by the warps that multiply (mma.sync): 42 and 74 us.
constexpr int kOuterThreads = 2 * kCopyThreads + 128 + 32;

template <int RT, bool SHARED>  // SHARED: a cluster shares an item
struct OuterTc {
  static constexpr int RP = RT * 16;
  static constexpr int kX = 2 * 64 * 128;             // two blocks of 64 columns
  static constexpr int kLow = RankRows<RT>::kBytes;   // one of the two numbers
  static constexpr int kStage = kX + 2 * kLow;
  static constexpr int kPitch = RP + 4;  // of the shares' sums, floats: rows a bank group apart
  static constexpr int kSums = SHARED ? 128 * kPitch * 4 : 0;
  // what two CTAs per SM leave room for, or one of the largest ranks
  static constexpr int kPerSm = RT == 8 || (RT == 4 && SHARED) ? 1 : 2;
  static constexpr int kStages = SHARED ? (RT == 1 ? 4 : RT == 2 ? 3 : RT == 4 ? 5 : 3)
                                        : (RT == 1 ? 5 : RT == 2 ? 4 : RT == 4 ? 3 : 4);
  static constexpr int kBytes = kStage * kStages + kSums + 1024;
  static constexpr uint32_t kCols = 2 * RP < 32 ? 32 : 2 * RP;
};

// Two neighbours of the gradient: columns c (and c + 1 in the rank-row form), rank rows r (and r + 1 otherwise).
template <bool BF16>
__device__ __forceinline__ void put_pair(uint16_t* out, const OuterParams& p, int rank, int c, int r, float a, float b) {
  const int64_t to = p.rank_rows ? static_cast<int64_t>(r) * p.len + c : static_cast<int64_t>(c) * rank + r;
  *reinterpret_cast<uint32_t*>(out + to) = Half<BF16>::put2(a, b);
}

template <bool BF16, int RT, bool SHARED>
__global__ void __launch_bounds__(kOuterThreads) outer_tc_kernel(LoraRows rows, OuterParams p0, OuterParams p1,
                                                                 int rank, int shares, int tiles0, int tiles, int items,
                                                                 uint32_t* err) {
  using L = OuterTc<RT, SHARED>;
  using R = RankRows<RT>;
  constexpr int S = L::kStages, RP = L::RP;
  extern __shared__ uint8_t raw[];
  __shared__ __align__(8) uint64_t full[S], empty[S], sums_full[2], sums_empty[2], top_ready[2], done;
  __shared__ uint32_t tmem_sh;
  __shared__ int abort_sh;
  __shared__ float top_sh[2], tops[4], leasts[4];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  const uint32_t base = smem_u32(sm);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int cs = SHARED ? shares : 1;
  const int crank = SHARED ? static_cast<int>(cluster_ctarank()) : 0;
  const int first = blockIdx.x / cs, stride = gridDim.x / cs;

  if (tid == 0) {
    for (int i = 0; i < S; ++i) {
      mbar_init(&full[i], 8);
      mbar_init(&empty[i], 1);
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
  volatile int* abort = &abort_sh;

  // an item's adapter, columns and steps; its rows are [r0, r1), this CTA's those from `begin` in n steps of 64
  struct Item {
    int which, c0, adapter, n, begin, r1;
  };
  auto item_at = [&](int it) {
    Item o;
    o.adapter = it / tiles;
    const int ct = it % tiles;
    o.which = ct < tiles0 ? 0 : 1;
    o.c0 = (ct < tiles0 ? ct : ct - tiles0) * 128;
    const int r0 = offset_at(rows, o.adapter);
    o.r1 = max(offset_at(rows, o.adapter + 1), r0);
    const int steps = o.r1 > r0 ? (o.r1 - r0 - 1) / 64 + 1 : 0;
    const int s0 = static_cast<int>(static_cast<int64_t>(steps) * crank / cs);
    o.begin = r0 + s0 * 64;
    o.n = static_cast<int>(static_cast<int64_t>(steps) * (crank + 1) / cs) - s0;
    return o;
  };

  // The copies of a step.  x: chunk tid % 16 (16 bytes) of rows tid / 16 + 8 i.  A warp has the sixteen rows
  // 2 * warp + {0, 1} + 8 i; lane j holds the number of row j % 2 + 8 (j / 2) of
  // them, loaded a step ahead.
  const int xc = tid & 15, xr = (tid >> 4) & 7;
  const uint32_t xto = (xc >> 3) * 8192 + swizzled<128>(xr, xc & 7);
  int number = -1;
  auto find = [&](const Item& o, int i) {
    const int place = o.begin + i * 64 + 2 * (warp & 3) + (lane & 1) + 8 * ((lane & 15) >> 1);
    number = i < o.n && place < o.r1 ? rows.source[place] : -1;
  };
  auto copy_x = [&](const Item& o, int st) {
    const OuterParams& p = o.which == 0 ? p0 : p1;
    const uint32_t to = base + st * L::kStage + xto;
    const bool in = o.c0 + xc * 8 < p.len;
    const uint16_t* x = p.x.p + o.c0 + xc * 8;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int v = __shfl_sync(0xffffffffu, number, (lane >> 4) + 2 * i);
      const bool has = in && v >= 0 && v < rows.m;
      cp16(to + i * 1024, has ? x + v * p.x.ld : p.x.p, has);
    }
  };
  // low: 16-byte chunk at % (4 RT) of row at / (4 RT), both numbers of a row side by side
  constexpr int kLowChunks = 2 * RT;  // per thread
  auto low_from = [&](const Item& o, int i, int j, bool& has) {
    const int at = (tid & 127) + j * kCopyThreads, r = at / (4 * RT), c = at % (4 * RT);
    const int place = o.begin + i * 64 + r;
    has = i < o.n && place < o.r1;
    const uint16_t* low = (o.which == 0 ? p0 : p1).low.low;
    return has ? low + static_cast<int64_t>(place) * (2 * RP) + c * 8 : low;
  };
  auto low_to = [&](int st, int j) {
    const int at = (tid & 127) + j * kCopyThreads, r = at / (4 * RT), c = at % (4 * RT);
    return st * L::kStage + L::kX + c / (2 * RT) * L::kLow + R::at(r, c % (2 * RT));
  };
  auto copy_low = [&](const Item& o, int i, int st) {  // bfloat16
#pragma unroll
    for (int j = 0; j < kLowChunks; ++j) {
      bool has;
      const uint16_t* from = low_from(o, i, j, has);
      cp16(base + low_to(st, j), from, has);
    }
  };
  uint4 held[BF16 ? 1 : kLowChunks];  // float16: the next step's low, and its rows' powers of two
  float held_by[BF16 ? 1 : kLowChunks];
  auto load_low = [&](const Item& o, int i) {
#pragma unroll
    for (int j = 0; j < (BF16 ? 0 : kLowChunks); ++j) {
      bool has;
      const uint16_t* from = low_from(o, i, j, has);
      held[j] = has ? *reinterpret_cast<const uint4*>(from) : make_uint4(0, 0, 0, 0);
      held_by[j] =
          has ? (o.which == 0 ? p0 : p1).low.factor[o.begin + i * 64 + ((tid & 127) + j * kCopyThreads) / (4 * RT)] : 0.f;
    }
  };
  // The rows' powers of two beside the largest are exact in 16 bits down to 2^-24.  (A row of kNoValue has nothing
  // but zeros, infinities and NaN: any power but zero will do.)
  auto store_low = [&](int st, float below) {
#pragma unroll
    for (int j = 0; j < (BF16 ? 0 : kLowChunks); ++j) {
      const __half2 by = __float2half2_rn(fmaxf(held_by[j] * below, 0x1p-24f));
      uint32_t w[4] = {held[j].x, held[j].y, held[j].z, held[j].w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const __half2 v = __hmul2(*reinterpret_cast<__half2*>(&w[k]), by);
        w[k] = *reinterpret_cast<const uint32_t*>(&v);
      }
      *reinterpret_cast<uint4*>(sm + low_to(st, j)) = make_uint4(w[0], w[1], w[2], w[3]);
    }
  };
  // An item with rows further apart: multiplied in 32 bits, each number rounded once.  From memory again and not
  // unrolled, since it is rare: unrolled beside the above it took a tenth of the gradients' time at rank 128.
  auto store_far = [&](const Item& o, int i, int st, float below) {
#pragma unroll 1
    for (int j = 0; j < (BF16 ? 0 : kLowChunks); ++j) {
      bool has;
      const uint16_t* from = low_from(o, i, j, has);
      uint4 u = make_uint4(0, 0, 0, 0);
      float by = 0.f;
      if (has) {
        u = *reinterpret_cast<const uint4*>(from);
        by = fmaxf((o.which == 0 ? p0 : p1).low.factor[o.begin + i * 64 + ((tid & 127) + j * kCopyThreads) / (4 * RT)] * below,
                   0x1p-126f);
      }
      uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[k]));
        const __half2 v = __floats2half2_rn(f.x * by, f.y * by);
        w[k] = *reinterpret_cast<const uint32_t*>(&v);
      }
      *reinterpret_cast<uint4*>(sm + low_to(st, j)) = make_uint4(w[0], w[1], w[2], w[3]);
    }
  };

  if (SHARED) cluster_arrive();
  pdl_wait();
  pdl_trigger();
  if (warp == 8) {
    tmem_alloc(&tmem_sh, L::kCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (SHARED) cluster_wait();  // the others have begun
  const uint32_t tmem = tmem_sh;

  if (warp < 4) {
    // ---------------------------------------------------------------- rows of x
    int g = 0;
    bool live = true;
    for (int it = first; it < items && live; it += stride) {
      const Item o = item_at(it);
      find(o, 0);
      for (int i = 0; i < o.n; ++i, ++g) {
        const int st = g % S;
        if (g >= S && !warp_wait(&empty[st], ((g / S) & 1) ^ 1, abort, err, kDevTimeoutProducer)) {
          live = false;
          break;
        }
        copy_x(o, st);
        find(o, i + 1);
        hand_over(&full[st]);
      }
    }
    copies_landed();
  } else if (warp >= 9) {
    // ---------------------------------------------------------------- rows of low
    // (after a wait that gave up these warps still go through the items, for the barriers among them)
    const int t = tid & 127;
    int g = 0, k = 0;
    bool live = true;
    for (int it = first; it < items; it += stride, ++k) {
      const Item o = item_at(it);
      float below = 1.f;
      bool far = false;
      if constexpr (!BF16) {
        // the largest power of two of this CTA's rows, and the smallest (kNoValue aside)
        const float* factor = (o.which == 0 ? p0 : p1).low.factor + o.begin;
        const int n = min(o.n * 64, o.r1 - o.begin);
        float top = 0.f, least = 0x1p127f;
        for (int r = t; r < n; r += kCopyThreads) {
          const float f = factor[r];
          top = fmaxf(top, f);
          least = fminf(least, f > kNoValue ? f : 0x1p127f);
        }
#pragma unroll
        for (int s = 16; s > 0; s >>= 1) {
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, s));
          least = fminf(least, __shfl_xor_sync(0xffffffffu, least, s));
        }
        named_bar_sync(1, kCopyThreads);  // the last item's are read
        if (lane == 0) tops[warp & 3] = top, leasts[warp & 3] = least;
        named_bar_sync(1, kCopyThreads);
        top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]));
        least = fminf(fminf(leasts[0], leasts[1]), fminf(leasts[2], leasts[3]));
        far = least < top * 0x1p-24f;
        if (!(top > 0.f)) top = 1.f;  // no rows
        below = 1.f / top;            // of a power of two: exact
        // the maximum of two items ago has been read when its sums have
        live = live && (k < 2 || warp_wait(&sums_empty[k & 1], ((k / 2) & 1) ^ 1, abort, err, kDevTimeoutDequant));
        if (live && t == 0) {
          top_sh[k & 1] = top;
          mbar_arrive(&top_ready[k & 1]);
        }
        load_low(o, 0);
      }
      for (int i = 0; i < o.n; ++i, ++g) {
        const int st = g % S;
        live = live && (g < S || warp_wait(&empty[st], ((g / S) & 1) ^ 1, abort, err, kDevTimeoutProducer));
        if (!live) continue;
        if constexpr (BF16) {
          copy_low(o, i, st);
        } else {
          if (far)
            store_far(o, i, st, below);
          else
            store_low(st, below);
          load_low(o, i + 1);
        }
        hand_over(&full[st]);
      }
    }
    copies_landed();
  } else if (warp == 8) {
    // ---------------------------------------------------------------- MMAs
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
        if (!stage_wait(&full[st], (g / S) & 1, abort, err)) {
          live = false;
          break;
        }
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
  } else {
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
      // a cluster's CTA c writes the columns from c * 128 / cs: the others' sums of them go to its shared
      // memory, [CTA][column][kPitch]
      const int own = 128 / cs;
      uint32_t sums = smem_u32(sm + L::kStage * S) + (crank * own + col % own) * L::kPitch * 4;
      if (SHARED) sums = mapa_shared(sums, col / own);
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
        if (SHARED) {
#pragma unroll
          for (int i = 0; i < 16; i += 4)
            st_cluster_f32x4(sums + (c + i) * 4, __uint_as_float(v[i]) * top, __uint_as_float(v[i + 1]) * top,
                             __uint_as_float(v[i + 2]) * top, __uint_as_float(v[i + 3]) * top);
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
  if (warp == 8) {
    tc_fence_after();
    tmem_dealloc(tmem, L::kCols);
  }
  if constexpr (SHARED) {
    cluster_arrive();
    cluster_wait();
    const int ct = first % tiles, own = 128 / cs;
    const OuterParams& p = ct < tiles0 ? p0 : p1;
    const int c0 = (ct < tiles0 ? ct : ct - tiles0) * 128 + crank * own;
    uint16_t* out = p.out + static_cast<int64_t>(first / tiles) * rank * p.len;
    const float* sums = reinterpret_cast<const float*>(sm + L::kStage * S);
    // two neighbours of the result per thread
    for (int at = tid; at < own * rank / 2; at += kOuterThreads) {
      const int half = (p.rank_rows ? own : rank) / 2;
      const int c = p.rank_rows ? at % half * 2 : at / half, r = p.rank_rows ? at / half : at % half * 2;
      if (c0 + c >= p.len) continue;
      const int step = p.rank_rows ? L::kPitch : 1;
      float a = 0.f, b = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j < cs) {
          const float* s = sums + (j * own + c) * L::kPitch + r;
          a += s[0];
          b += s[step];
        }
      put_pair<BF16>(out, p, rank, c0 + c, r, a, b);
    }
  }
}

// ------------------------------------------------------------------ launches
template <bool BF16, int RT, bool SHARED>
cudaError_t outer_as(const LoraRows& rows, const OuterParams (&p)[2], int rank, int cs, int tiles0, int tiles, int sms,
                     cudaStream_t s) {
  using L = OuterTc<RT, SHARED>;
  const int items = tiles * rows.adapters;
  const int grid = SHARED ? items * cs : std::min(items, L::kPerSm * sms);
  auto kernel = outer_tc_kernel<BF16, RT, SHARED>;
  if (const cudaError_t e = allow_smem(kernel, L::kBytes); e != cudaSuccess) return e;
  return launch_pdl(kernel, dim3(static_cast<unsigned>(grid)), dim3(kOuterThreads), L::kBytes, cs, s, rows, p[0], p[1],
                    rank, cs, tiles0, tiles, items, device_error_word());
}

template <bool BF16, int RT>
cudaError_t outer_plan(const LoraRows& rows, const OuterParams (&p)[2], int rank, int sms, cudaStream_t s) {
  const int t0 = (p[0].len + 127) / 128, tiles = t0 + (p[1].len + 127) / 128;
  // shares of an adapter's rows: as many as there is room for at once, each of 128 rows or more on average
  const int64_t room = static_cast<int64_t>(OuterTc<RT, true>::kPerSm) * sms;
  int cs = 1;
  while (cs < 8 && static_cast<int64_t>(tiles) * rows.adapters * cs * 2 <= room && rows.m / rows.adapters >= 256 * cs)
    cs *= 2;
  return cs > 1 ? outer_as<BF16, RT, true>(rows, p, rank, cs, t0, tiles, sms, s)
                : outer_as<BF16, RT, false>(rows, p, rank, 1, t0, tiles, sms, s);
}

}  // namespace

cudaError_t launch_lora_outer(const LoraRows& rows, const OuterParams (&p)[2], int rank, bool bf16, int sms,
                              cudaStream_t s) {
  return with_rank(rank, [&](auto rt) {
    constexpr int RT = decltype(rt)::value;
    return bf16 ? outer_plan<true, RT>(rows, p, rank, sms, s) : outer_plan<false, RT>(rows, p, rank, sms, s);
  });
}

}  // namespace wqmm
