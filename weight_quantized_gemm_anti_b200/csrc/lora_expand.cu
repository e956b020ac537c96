// lora_expand.cu -- the low-rank adapters' contraction over the rank, out = y + low W^T.
#include "lora_tc.cuh"

namespace wqmm {
namespace {

// ------------------------------------------------------------------ expand
// A CTA has BM rows and `chunks` times 128 columns.  A row's low values stay in
// registers as the matrix instruction's first operand; the weights of 128
// columns are staged in shared memory, the next ones while these are used.
// The weights' columns are dealt to the instruction's tiles of eight such that
// a thread's four results of a 32-column group are neighbours with the next
// three tiles': column q * 8 + 2 j + e of the group is column 2 q + e of tile
// j, so a thread adds and stores 16 bytes of a row at once, four threads 64.
// Results leave the registers that the instruction wrote, with no detour through
// shared memory.  Up to rank 32, where the products take a fifth of the time that y
// and the result need, or few rows; the rest below.  4096 x 4096, rank 16, 67 MB:
// about 14 us (the memory's floor is 10.4).
template <int RT, bool KM>
struct ExpandSmem {
  static constexpr int RP = RT * 16;
  static constexpr int kPitch = KM ? RP * 2 + 16 : 256 + 16;
  static constexpr int kBuf = (KM ? 128 : RP) * kPitch;
  static constexpr int kBytes = 2 * kBuf;
};

template <bool BF16, int RT, bool KM, int WM>
__global__ void __launch_bounds__(kThreads) expand_kernel(LoraRows rows, ExpandParams p, int rank, int chunks) {
  extern __shared__ __align__(128) uint8_t sm[];
  constexpr int RP = RT * 16, BM = WM * 16;
  constexpr int GROUPS = WM == 1 ? 1 : 4;  // 32-column groups of a chunk per warp
  using L = ExpandSmem<RT, KM>;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, q = lane & 3;
  const uint32_t base = smem_u32(sm);
  Tile tile;
  pdl_wait();
  pdl_trigger();
  if (!find_tile(rows, p.bare, BM, blockIdx.x, tile)) return;
  const bool with = tile.group < rows.adapters;
  const uint16_t* w = p.w + static_cast<int64_t>(with ? tile.group : 0) * rank * p.len;
  const int c_begin = blockIdx.y * chunks * 128;
  const int c_end = min(c_begin + chunks * 128, p.len);

  constexpr int WR = KM ? 1 : (RP * 4 + kThreads - 1) / kThreads;
  uint4 wr[WR][4];
  // k-major: copies under way in shared memory; rank-major: 64 bytes (32 columns) of a rank row per
  // thread and step, in registers until put() changes their words' places
  auto fetch = [&](int c0, int buf) {
    if constexpr (KM) {
      const uint32_t ws = base + buf * L::kBuf;
      constexpr int C = RP / 8;
#pragma unroll
      for (int i = 0; i < (128 * C + kThreads - 1) / kThreads; ++i) {
        const int at = tid + i * kThreads, col = at / C, c = at % C;
        const bool has = c0 + col < c_end && c * 8 < rank;
        // column (q, j, e) of its group of 32 goes to row (j, q, e)
        const int in = col & 31, to = (col & ~31) | (((in >> 1) & 3) << 3) | ((in >> 3) << 1) | (in & 1);
        cp16(ws + to * L::kPitch + c * 16, has ? w + static_cast<int64_t>(c0 + col) * rank + c * 8 : w, has);
      }
      cp_async_commit();
    } else {
#pragma unroll
      for (int i = 0; i < WR; ++i) {
        const int at = tid + i * kThreads, r = at / 4, col = c0 + (at % 4) * 32;
        const bool has = r < rank && r < RP && col < c_end;
#pragma unroll
        for (int j = 0; j < 4; ++j)
          wr[i][j] = has ? *reinterpret_cast<const uint4*>(w + static_cast<int64_t>(r) * p.len + col + j * 8)
                         : make_uint4(0, 0, 0, 0);
      }
    }
  };
  auto put = [&](int buf) {
    if constexpr (KM) {
      cp_async_wait_group<0>();
    } else {
#pragma unroll
      for (int i = 0; i < WR; ++i) {
        const int at = tid + i * kThreads, r = at / 4;
        if (r >= RP) break;
        const uint4* v = wr[i];
        uint8_t* o = sm + buf * L::kBuf + r * L::kPitch + (at % 4) * 64;
        *reinterpret_cast<uint4*>(o) = make_uint4(v[0].x, v[1].x, v[2].x, v[3].x);
        *reinterpret_cast<uint4*>(o + 16) = make_uint4(v[0].y, v[1].y, v[2].y, v[3].y);
        *reinterpret_cast<uint4*>(o + 32) = make_uint4(v[0].z, v[1].z, v[2].z, v[3].z);
        *reinterpret_cast<uint4*>(o + 48) = make_uint4(v[0].w, v[1].w, v[2].w, v[3].w);
      }
    }
  };
  if (with) fetch(c_begin, 0);

  // this thread's two rows: their places in y and out
  const int wrow = WM == 1 ? 0 : warp * 16;
  int row[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) row[i] = row_at(rows, tile.p0 + wrow + g + 8 * i, tile.p1);
  uint4 y[GROUPS][2], next[GROUPS][2];
  auto fetch_y = [&](int c0) {
#pragma unroll
    for (int s = 0; s < GROUPS; ++s)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int col = c0 + (WM == 1 ? warp : s) * 32 + q * 8;
        next[s][i] = make_uint4(0, 0, 0, 0);
        if (p.y.p && row[i] >= 0 && col < c_end)
          next[s][i] = *reinterpret_cast<const uint4*>(p.y.p + row[i] * p.y.ld + col);
      }
  };
  fetch_y(c_begin);

  float factor[2] = {1.f, 1.f};
  uint32_t a[2][RT][4];  // hi, lo
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int place = tile.p0 + wrow + g + 8 * i;
    const bool has = with && place < tile.p1;
    if (!BF16 && has) factor[i] = p.low.factor[place];
    const uint32_t* low = reinterpret_cast<const uint32_t*>(p.low.low + (has ? static_cast<int64_t>(place) * (2 * RP) : 0));
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int k = 0; k < RT; ++k) {
        a[h][k][i] = has ? low[h * (RP / 2) + k * 8 + q] : 0u;
        a[h][k][i + 2] = has ? low[h * (RP / 2) + k * 8 + 4 + q] : 0u;
      }
  }

  int buf = 0;
  for (int c0 = c_begin; c0 < c_end; c0 += 128, buf ^= 1) {
#pragma unroll
    for (int s = 0; s < GROUPS; ++s)
#pragma unroll
      for (int i = 0; i < 2; ++i) y[s][i] = next[s][i];
    if (c0 + 128 < c_end) fetch_y(c0 + 128);
    if (with) {
      put(buf);
      __syncthreads();  // this chunk's weights are there, and the other buffer is read no more
      if (c0 + 128 < c_end) fetch(c0 + 128, buf ^ 1);
    }
    const uint32_t ws = base + buf * L::kBuf;
#pragma unroll
    for (int s = 0; s < GROUPS; ++s) {
      const int grp = WM == 1 ? warp : s;
      float acc[4][4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[j][i] = 0.f;
      if (with) {
#pragma unroll
        for (int k = 0; k < RT; ++k)
#pragma unroll
          for (int j = 0; j < 4; j += 2) {
            uint32_t b[4];
            if constexpr (KM) {
              const int r = grp * 32 + j * 8 + ((lane >> 4) << 3) + (lane & 7), c = k * 2 + ((lane >> 3) & 1);
              ldsm4(b, ws + r * L::kPitch + c * 16);
            } else {
              const int r = k * 16 + (lane & 15), c = grp * 4 + j + (lane >> 4);
              ldsm4t(b, ws + r * L::kPitch + c * 16);
            }
#pragma unroll
            for (int h = 1; h >= 0; --h) {  // the small part first
              mma<BF16>(acc[j], a[h][k], b[0], b[1]);
              mma<BF16>(acc[j + 1], a[h][k], b[2], b[3]);
            }
          }
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int col = c0 + grp * 32 + q * 8;
        if (row[i] < 0 || col >= c_end) continue;
        const uint32_t yv[4] = {y[s][i].x, y[s][i].y, y[s][i].z, y[s][i].w};
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

// ------------------------------------------------------------------ larger ranks
// Above rank 32 the products are on the tensor cores' tcgen05 path: a CTA has
// 128 rows, whose low values stay in shared memory as two K-major operands (the
// two 16-bit numbers, MMAs into the same sums), and goes through 128 columns at a
// time.  The weights pass through registers, where their columns change places
// as above; rank-major ones are an MN-major operand.  The sums come back in the
// fragments of the matrix instruction (16 rows x 8 columns, four times), so a
// thread again adds and stores 16 bytes of a row at once.
// The products of a chunk run while the one before it is written.
// Bound by y and the result (8192 x 4096, the adapters' whole part, against the kernel above: rank 64
// 64 us and 75.6, rank 128 71 and 94.6; the gradient 122 and 142, 147 and 183).
constexpr int kExpandThreads = 256;

template <int RT>
struct ExpandTc {
  static constexpr int RP = RT * 16;
  static constexpr int kBlock = 128 * 128;  // 128 rows of 64 numbers
  static constexpr int kLow = 2 * RP / 64 * kBlock, kW = RP / 64 * kBlock;
  static constexpr int kBufs = RT == 4 ? 2 : 1;  // two CTAs per SM
  static constexpr int kBytes = kLow + kBufs * kW + 1024;
  static constexpr uint32_t kCols = 256;  // the sums of two chunks
};

// 16 lanes x 256 bit, four times: row g's columns 2 q, 2 q + 1 of eight in r[4 j], r[4 j + 1], row g + 8's behind.
__device__ __forceinline__ void tmem_ld_rows(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
      "%14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}

template <bool BF16, int RT, bool KM>
__global__ void __launch_bounds__(kExpandThreads, 2)
    expand_tc_kernel(LoraRows rows, ExpandParams p, int rank, int chunks, uint32_t* err) {
  using L = ExpandTc<RT>;
  constexpr int RP = L::RP;
  extern __shared__ uint8_t raw[];
  __shared__ __align__(8) uint64_t done[2];
  __shared__ uint32_t tmem_sh;
  __shared__ int abort_sh;
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  const uint32_t base = smem_u32(sm);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, q = lane & 3;
  const int quad = warp & 3, side = warp >> 2;  // 32 rows, 64 columns of a chunk
  volatile int* abort = &abort_sh;
  if (tid == 0) {
    mbar_init(&done[0], 1);
    mbar_init(&done[1], 1);
    abort_sh = 0;
    fence_barrier_init();
  }
  pdl_wait();
  pdl_trigger();
  Tile tile;
  if (!find_tile(rows, p.bare, 128, blockIdx.x, tile)) return;
  const bool with = tile.group < rows.adapters;
  const uint16_t* w = p.w + static_cast<int64_t>(with ? tile.group : 0) * rank * p.len;
  const int c_begin = blockIdx.y * chunks * 128;
  const int c_end = min(c_begin + chunks * 128, p.len);
  const int n = c_end > c_begin ? (c_end - c_begin + 127) / 128 : 0;

  // k-major: 16 bytes of a column's rank each; rank-major: 32 columns of a rank row, in four
  constexpr int WR = RT;
  uint4 wr[WR];
  auto fetch = [&](int c) {
    const int c0 = c_begin + c * 128;
#pragma unroll
    for (int i = 0; i < WR; ++i) {
      const uint16_t* from;
      bool has;
      if constexpr (KM) {
        const int at = tid + i * kExpandThreads, col = c0 + at / (RP / 8), k = at % (RP / 8) * 8;
        has = c < n && col < c_end && k < rank;
        from = w + static_cast<int64_t>(col) * rank + k;
      } else {
        const int at = tid + i / 4 * kExpandThreads, k = at / 4, col = c0 + at % 4 * 32;
        has = c < n && col < c_end && k < rank;
        from = w + static_cast<int64_t>(k) * p.len + col + i % 4 * 8;
      }
      wr[i] = has ? *reinterpret_cast<const uint4*>(from) : make_uint4(0, 0, 0, 0);
    }
  };
  auto put = [&](int c) {
    uint8_t* ws = sm + L::kLow + c % L::kBufs * L::kW;
    if constexpr (KM) {
#pragma unroll
      for (int i = 0; i < WR; ++i) {
        const int at = tid + i * kExpandThreads, col = at / (RP / 8), k = at % (RP / 8);
        const int in = col & 31, to = (col & ~31) | (((in >> 1) & 3) << 3) | ((in >> 3) << 1) | (in & 1);
        *reinterpret_cast<uint4*>(ws + k / 8 * L::kBlock + swizzled<128>(to, k % 8)) = wr[i];
      }
    } else {
#pragma unroll
      for (int i = 0; i < WR; i += 4) {
        const int at = tid + i / 4 * kExpandThreads, k = at / 4, c32 = at % 4;
        uint8_t* o = ws + c32 / 2 * (RP * 128);
        const int b = c32 % 2 * 4;
        const uint4 v0 = wr[i], v1 = wr[i + 1], v2 = wr[i + 2], v3 = wr[i + 3];
        *reinterpret_cast<uint4*>(o + swizzled<128>(k, b)) = make_uint4(v0.x, v1.x, v2.x, v3.x);
        *reinterpret_cast<uint4*>(o + swizzled<128>(k, b + 1)) = make_uint4(v0.y, v1.y, v2.y, v3.y);
        *reinterpret_cast<uint4*>(o + swizzled<128>(k, b + 2)) = make_uint4(v0.z, v1.z, v2.z, v3.z);
        *reinterpret_cast<uint4*>(o + swizzled<128>(k, b + 3)) = make_uint4(v0.w, v1.w, v2.w, v3.w);
      }
    }
  };
  if (with) {
    if (warp == 0) {
      tmem_alloc(&tmem_sh, L::kCols);
      tmem_relinquish();
    }
    fetch(0);
    // the rows' low values, both numbers side by side
    constexpr int C = RP / 4;
#pragma unroll 4
    for (int at = tid; at < 128 * C; at += kExpandThreads) {
      const int r = at / C, c = at % C, place = tile.p0 + r;
      const bool has = place < tile.p1;
      cp16(base + c / 8 * L::kBlock + swizzled<128>(r, c % 8),
           has ? p.low.low + static_cast<int64_t>(place) * (2 * RP) + c * 8 : p.low.low, has);
    }
    cp_async_commit();
  }

  // this thread's rows: their places in y and out
  int row[4];
  float factor[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int place = tile.p0 + quad * 32 + g + 8 * i;
    row[i] = row_at(rows, place, tile.p1);
    factor[i] = !BF16 && with && place < tile.p1 ? p.low.factor[place] : 1.f;
  }
  uint4 y[2][4];
  auto fetch_y = [&](int c, int s, int i) {
    const int col = c_begin + c * 128 + side * 64 + s * 32 + q * 8;
    y[s][i] = p.y.p && row[i] >= 0 && col < c_end
                  ? *reinterpret_cast<const uint4*>(p.y.p + row[i] * p.y.ld + col)
                  : make_uint4(0, 0, 0, 0);
  };
#pragma unroll
  for (int s = 0; s < 2; ++s)
#pragma unroll
    for (int i = 0; i < 4; ++i) fetch_y(0, s, i);

  uint32_t tmem = 0;
  auto multiply = [&](int c) {  // the first warp
    constexpr uint32_t kIdesc = idesc_make(1u, BF16 ? 1u : 0u, 128, 128) | (KM ? 0u : kBMn);
    constexpr uint64_t kKBits = operand_bits(128, 16, 1024), kMnBits = operand_bits(128, RP * 128, 1024);
    const uint32_t ws = base + L::kLow + c % L::kBufs * L::kW;
    fence_proxy_async_smem();
    tc_fence_after();
    if (elect_one()) {
#pragma unroll
      for (int h = 1; h >= 0; --h)  // the small part first
#pragma unroll
        for (int k = 0; k < RT; ++k)
          mma_f16_ss(tmem + (c & 1) * 128,
                     operand(base + (h * (RP / 64) + k / 4) * L::kBlock + k % 4 * 32, kKBits),
                     KM ? operand(ws + k / 4 * L::kBlock + k % 4 * 32, kKBits) : operand(ws + k * 2048, kMnBits),
                     kIdesc, h < 1 || k > 0);
      mma_commit(&done[c & 1]);
    }
    __syncwarp();
  };
  // the next chunk's weights into shared memory and its products under way (every thread comes here)
  auto begin = [&](int c) {
    put(c);
    cp_async_wait_group<0>();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (c == 0) tmem = tmem_sh;
    if (warp == 0) multiply(c);
    fetch(c + 1);
  };
  bool live = true;
  auto finished = [&](int c) {
    live = warp_wait(&done[c & 1], (c >> 1) & 1, abort, err, kDevTimeoutEpilogue) && live;
    tc_fence_after();
  };
  if (with && n > 0) begin(0);
  for (int c = 0; c < n; ++c) {
    if (with) {
      // one buffer of weights: free when the last products are done
      if (L::kBufs == 1) finished(c);
      if (c + 1 < n) begin(c + 1);
      if (L::kBufs == 2) finished(c);
    }
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t v[16];
        if (with) {
          tmem_ld_rows(tmem + (static_cast<uint32_t>(quad * 32 + h * 16) << 16) + (c & 1) * 128 + side * 64 + s * 32, v);
          tmem_wait_ld_r16(v);
        }
        const int col = c_begin + c * 128 + side * 64 + s * 32 + q * 8;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int i = 2 * h + e;
          const uint32_t yv[4] = {y[s][i].x, y[s][i].y, y[s][i].z, y[s][i].w};
          uint32_t o[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            o[j] = yv[j];
            if (with) {
              float v0 = __uint_as_float(v[j * 4 + 2 * e]), v1 = __uint_as_float(v[j * 4 + 2 * e + 1]);
              const float y0 = Half<BF16>::get(yv[j] & 0xffff), y1 = Half<BF16>::get(yv[j] >> 16);
              v0 = BF16 ? v0 + y0 : fmaf(factor[i], v0, y0);
              v1 = BF16 ? v1 + y1 : fmaf(factor[i], v1, y1);
              o[j] = Half<BF16>::put2(v0, v1);
            }
          }
          if (live && row[i] >= 0 && col < c_end)
            *reinterpret_cast<uint4*>(p.out + row[i] * p.ldo + col) = make_uint4(o[0], o[1], o[2], o[3]);
          fetch_y(c + 1, s, i);
        }
      }
  }
  if (!with) return;  // the same for the whole CTA
  // after a wait that gave up, the products under way first
  if (warp == 0 && !live && n > 0) {
    volatile int no_abort = 0;
    warp_wait(&done[(n - 1) & 1], ((n - 1) >> 1) & 1, &no_abort, err, kDevTimeoutDrain);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem_sh, L::kCols);
  }
}

template <bool BF16, int RT, bool KM>
cudaError_t expand_tc_as(const LoraRows& rows, const ExpandParams& p, int rank, int sms, cudaStream_t s) {
  const int64_t tiles = most_tiles(rows.m, rows.adapters + p.bare, 128);
  const int all = (p.len + 127) / 128;
  int chunks = 8;
  while (chunks > 1 && tiles * ((all + chunks - 1) / chunks) < 2 * sms) chunks /= 2;
  auto kernel = expand_tc_kernel<BF16, RT, KM>;
  const size_t smem = ExpandTc<RT>::kBytes;
  if (const cudaError_t e = allow_smem(kernel, smem); e != cudaSuccess) return e;
  return launch_pdl(kernel, dim3(static_cast<unsigned>(tiles), static_cast<unsigned>((all + chunks - 1) / chunks)),
                    dim3(kExpandThreads), smem, 1, s, rows, p, rank, chunks, device_error_word());
}

template <bool BF16, int RT, bool KM, int WM>
cudaError_t expand_as(const LoraRows& rows, const ExpandParams& p, int rank, int sms, cudaStream_t s) {
  constexpr int BM = WM * 16;
  const int64_t tiles = most_tiles(rows.m, rows.adapters + p.bare, BM);
  // columns per CTA: up to 1024, fewer where there would be under two CTAs per SM (4096 x 4096, rank 16: two
  // CTAs 28.5 us with a contraction before, eight 30.1), or eight of the short-lived ones of few rows
  const int all = (p.len + 127) / 128;
  int chunks = 8;
  while (chunks > 1 && tiles * ((all + chunks - 1) / chunks) < (WM == 1 ? 8 : 2) * sms) chunks /= 2;
  auto kernel = expand_kernel<BF16, RT, KM, WM>;
  const size_t smem = ExpandSmem<RT, KM>::kBytes;
  if (const cudaError_t e = allow_smem(kernel, smem); e != cudaSuccess) return e;
  return launch_pdl(kernel, dim3(static_cast<unsigned>(tiles), static_cast<unsigned>((all + chunks - 1) / chunks)),
                    dim3(kThreads), smem, 1, s, rows, p, rank, chunks);
}

}  // namespace

cudaError_t launch_lora_expand(const LoraRows& rows, const ExpandParams& p, int rank, bool rank_major, bool bf16,
                               int sms, cudaStream_t s) {
  return with_rank(rank, [&](auto rt) {
    constexpr int RT = decltype(rt)::value;
    auto pick = [&](auto t, auto km) {
      constexpr bool T = decltype(t)::value, KM = decltype(km)::value;
      if constexpr (!KM)  // few rows of a forward pass: lora_few.cu
        if (few_rows(rows, rank)) return expand_as<T, RT, false, 1>(rows, p, rank, sms, s);
      if constexpr (RT >= 4) return expand_tc_as<T, RT, KM>(rows, p, rank, sms, s);
      else if constexpr (!KM || RT > 1) return expand_as<T, RT, KM, 4>(rows, p, rank, sms, s);
      return cudaErrorInvalidValue;  // a forward pass at rank 16: lora_few.cu
    };
    auto by_major = [&](auto t) { return rank_major ? pick(t, std::false_type()) : pick(t, std::true_type()); };
    return bf16 ? by_major(std::true_type()) : by_major(std::false_type());
  });
}

}  // namespace wqmm
