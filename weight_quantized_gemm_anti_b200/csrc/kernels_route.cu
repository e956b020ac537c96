// kernels_route.cu -- tokens sorted by expert and back: a stable counting sort
// of the expert ids, the copy of the tokens into that order, the weighted sum
// of the experts' rows in token order, and that sum's gradient.
//
// All four move every byte they need once and compute next to nothing, so
// memory bounds them (the launch, at a few tokens).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "launch.cuh"
#include "route.h"

namespace wqmm {
namespace {

// ------------------------------------------------------------------ counting sort
// Position of slot i = (slots of lower groups) + (slots before i of its own
// group).  The slots are cut into chunks, one CTA each, and a chunk into one
// run per warp; counts per (chunk, group) and per (warp, group) give each run
// its first position in every group, and inside a run a warp goes through its
// slots 32 at a time, the lanes of one group ranked by lane.  Every count is a
// whole number added in a fixed place, so the order is stable and the same in
// every run.  Ids outside [0, groups) make one more group, behind the others.
constexpr int kBatch = 4;        // slots per lane
constexpr int kSortCluster = 8;  // CTAs

// The lanes whose group is this lane's (groups are below 2^bits): one vote per
// bit.  4096 slots in 256 groups, sorted by one CTA, took 8.4 us with it and 11.9 us
// with __match_any_sync.
__device__ __forceinline__ uint32_t same_group(int e, int bits) {
  uint32_t same = 0xffffffffu;
  for (int b = 0; b < bits; ++b) {
    const uint32_t set = __ballot_sync(0xffffffffu, (e >> b) & 1);
    same &= ((e >> b) & 1) ? set : ~set;
  }
  return same;
}

template <typename IdT>
__device__ __forceinline__ int group_of(const IdT* ids, int64_t i, int groups) {
  const IdT v = ids[i];
  return (v >= 0 && v < static_cast<IdT>(groups)) ? static_cast<int>(v) : groups;
}

// A cluster neighbour's copy of a shared variable.
__device__ __forceinline__ int load_of_cta(const int* mine, int cta) {
  const uint32_t at = static_cast<uint32_t>(__cvta_generic_to_shared(mine));
  uint32_t there;
  int v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(there) : "r"(at), "r"(cta));
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(there) : "memory");
  return v;
}

template <typename IdT>
__global__ void __launch_bounds__(256) sort_count_kernel(SortParams p) {
  extern __shared__ int count[];
  for (int e = threadIdx.x; e <= p.groups; e += blockDim.x) count[e] = 0;
  pdl_wait();
  pdl_trigger();
  __syncthreads();
  const IdT* ids = static_cast<const IdT*>(p.ids);
  const int64_t lo = static_cast<int64_t>(blockIdx.x) * p.chunk;
  const int64_t hi = min(lo + p.chunk, p.slots);
  for (int64_t i = lo + threadIdx.x; i < hi; i += blockDim.x) atomicAdd(&count[group_of(ids, i, p.groups)], 1);
  __syncthreads();
  for (int e = threadIdx.x; e <= p.groups; e += blockDim.x)
    p.hist[static_cast<int64_t>(blockIdx.x) * (p.groups + 1) + e] = count[e];
}

// CLUSTER: the chunks' CTAs are one cluster and read each other's counts in
// shared memory; otherwise the counts of all chunks are in hist, from the kernel
// above (or there is one chunk).
// Shared memory: next[warps][groups + 1], total[groups + 1], count[groups + 1], the scan's warp sums [32].
template <typename IdT, bool CLUSTER>
__global__ void __launch_bounds__(1024) sort_place_kernel(SortParams p) {
  extern __shared__ int sm[];
  const int warps = blockDim.x >> 5, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int buckets = p.groups + 1;
  int* next = sm;
  int* total = sm + warps * buckets;
  int* count = total + buckets;
  int* sums = count + buckets;
  for (int i = threadIdx.x; i < warps * buckets; i += blockDim.x) next[i] = 0;
  pdl_wait();
  pdl_trigger();
  __syncthreads();

  const IdT* ids = static_cast<const IdT*>(p.ids);
  const int64_t lo = static_cast<int64_t>(blockIdx.x) * p.chunk;
  const int64_t hi = min(lo + p.chunk, p.slots);
  const int run = ((p.chunk + warps - 1) / warps + 31) & ~31;
  const int64_t r0 = min(lo + static_cast<int64_t>(warp) * run, hi), r1 = min(r0 + run, hi);
  int* mine = next + warp * buckets;
  // The ids of a batch are loaded together, so that their latency is paid once;
  // a run of one batch keeps what it has for the second walk.
  // A lane behind the run's end has the group `buckets`, which is not counted.
  const int bits = 32 - __clz(buckets);
  int group[kBatch];
  uint32_t same[kBatch];
  auto load = [&](int64_t i0) {
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const int64_t i = i0 + b * 32 + lane;
      group[b] = i < r1 ? group_of(ids, i, p.groups) : buckets;
    }
#pragma unroll
    for (int b = 0; b < kBatch; ++b) same[b] = same_group(group[b], bits);
  };
  for (int64_t i0 = r0; i0 < r1; i0 += 32 * kBatch) {
    load(i0);
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      if (group[b] < buckets && lane == __ffs(same[b]) - 1) mine[group[b]] += __popc(same[b]);
      __syncwarp();
    }
  }
  __syncthreads();

  if constexpr (CLUSTER) {
    for (int e = threadIdx.x; e < buckets; e += blockDim.x) {
      int all = 0;
      for (int w = 0; w < warps; ++w) all += next[w * buckets + e];
      count[e] = all;
    }
    cluster_arrive();
    cluster_wait();
  }
  // per group: the runs' counts become first places within the chunk's slots of
  // the group, behind those of earlier chunks
  for (int e = threadIdx.x; e < buckets; e += blockDim.x) {
    int before = 0, all = 0;
    if constexpr (CLUSTER) {
      int n[8];
#pragma unroll
      for (int c = 0; c < 8; ++c) n[c] = c < p.chunks ? load_of_cta(count + e, c) : 0;
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        all += n[c];
        before += c < static_cast<int>(blockIdx.x) ? n[c] : 0;
      }
    } else if (p.chunks > 1) {
#pragma unroll 8
      for (int c = 0; c < p.chunks; ++c) {
        const int n = p.hist[static_cast<int64_t>(c) * buckets + e];
        all += n;
        before += c < static_cast<int>(blockIdx.x) ? n : 0;
      }
    }
    for (int w = 0; w < warps; ++w) {
      const int n = next[w * buckets + e];
      next[w * buckets + e] = before;
      before += n;
    }
    total[e] = p.chunks > 1 ? all : before;
  }
  if constexpr (CLUSTER) cluster_arrive();  // this CTA has read the others' counts
  __syncthreads();

  // exclusive scan of total over the groups: consecutive ones per thread
  const int per = (buckets + blockDim.x - 1) / blockDim.x;
  const int e0 = min(static_cast<int>(threadIdx.x) * per, buckets), e1 = min(e0 + per, buckets);
  int own = 0;
  for (int e = e0; e < e1; ++e) own += total[e];
  int upto = own;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, upto, d);
    if (lane >= d) upto += v;
  }
  if (lane == 31) sums[warp] = upto;
  __syncthreads();
  if (warp == 0) {
    int v = lane < warps ? sums[lane] : 0;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, v, d);
      if (lane >= d) v += u;
    }
    if (lane < warps) sums[lane] = v;
  }
  __syncthreads();
  int at = upto - own + (warp > 0 ? sums[warp - 1] : 0);
  for (int e = e0; e < e1; ++e) {
    const int n = total[e];
    total[e] = at;
    if (blockIdx.x == 0) p.offsets[e] = at;
    at += n;
  }
  __syncthreads();

  for (int64_t i0 = r0; i0 < r1; i0 += 32 * kBatch) {
    if (r1 - r0 > 32 * kBatch) load(i0);
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const int e = group[b];
      if (e < buckets) {
        const int64_t i = i0 + b * 32 + lane;
        const int place = total[e] + mine[e] + __popc(same[b] & ((1u << lane) - 1));
        p.source[place] = static_cast<int>(i);
        p.position[i] = e < p.groups ? place : -1;
      }
      __syncwarp();
      if (e < buckets && lane == __ffs(same[b]) - 1) mine[e] += __popc(same[b]);
      __syncwarp();
    }
  }
  if constexpr (CLUSTER) cluster_wait();  // the others have read this CTA's
}

// ------------------------------------------------------------------ vectors
template <int BYTES>
struct RawVec;
template <>
struct RawVec<16> { using T = uint4; };
template <>
struct RawVec<8> { using T = uint2; };
template <>
struct RawVec<4> { using T = uint32_t; };
template <>
struct RawVec<2> { using T = uint16_t; };
template <>
struct RawVec<1> { using T = uint8_t; };

template <int TYPE>
struct Elem;
template <>
struct Elem<kRtF16> {
  using T = __half;
  static __device__ __forceinline__ float get(T v) { return __half2float(v); }
  static __device__ __forceinline__ T put(float v) { return __float2half_rn(v); }
};
template <>
struct Elem<kRtBf16> {
  using T = __nv_bfloat16;
  static __device__ __forceinline__ float get(T v) { return __bfloat162float(v); }
  static __device__ __forceinline__ T put(float v) { return __float2bfloat16_rn(v); }
};
template <>
struct Elem<kRtF32> {
  using T = float;
  static __device__ __forceinline__ float get(T v) { return v; }
  static __device__ __forceinline__ T put(float v) { return v; }
};

template <int TYPE, int N>
struct Pack {
  using E = Elem<TYPE>;
  union {
    typename RawVec<N * sizeof(typename E::T)>::T raw;
    typename E::T v[N];
  };
  __device__ __forceinline__ Pack() {}
};

__device__ __forceinline__ float load_scalar(const void* p, int64_t i, int type) {
  if (type == kRtF32) return static_cast<const float*>(p)[i];
  if (type == kRtBf16) return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
  return __half2float(static_cast<const __half*>(p)[i]);
}

__device__ __forceinline__ void store_scalar(void* p, int64_t i, int type, float v) {
  if (type == kRtF32)
    static_cast<float*>(p)[i] = v;
  else if (type == kRtBf16)
    static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
  else
    static_cast<__half*>(p)[i] = __float2half_rn(v);
}

// ------------------------------------------------------------------ dispatch
// A token's row is read once and written to each of its positions: no row is
// read again from memory, and all writes are whole rows.  `tpt` threads share a
// row, each UN vectors of it (four where there is work for every thread of the
// device four times over, one otherwise).  8192 tokens of 8192 bfloat16, four
// choices: 672 MB in 104 us, the rate of a plain copy; 16 tokens: the launch.
template <int VB, int UN>
__global__ void __launch_bounds__(256) dispatch_kernel(DispatchParams p, int tpt) {
  using V = typename RawVec<VB>::T;
  pdl_wait();
  pdl_trigger();
  const int64_t t = static_cast<int64_t>(blockIdx.x) * (blockDim.x / tpt) + threadIdx.x / tpt;
  if (t >= p.tokens) return;
  const int64_t nv = p.row_bytes / VB;
  const int64_t c0 = static_cast<int64_t>(blockIdx.y) * tpt * UN + threadIdx.x % tpt;
  const V* x = reinterpret_cast<const V*>(p.x) + t * nv;
  V v[UN];
#pragma unroll
  for (int u = 0; u < UN; ++u)
    if (c0 + u * tpt < nv) v[u] = x[c0 + u * tpt];
  for (int j = 0; j < p.top; ++j) {
    const int64_t pos = p.position[t * p.top + j];
    if (pos < 0 || pos >= p.rows) continue;
    V* o = reinterpret_cast<V*>(p.out) + pos * nv;
#pragma unroll
    for (int u = 0; u < UN; ++u)
      if (c0 + u * tpt < nv) o[c0 + u * tpt] = v[u];
  }
}

// ------------------------------------------------------------------ combine
// Sums in 32 bits, in the order of the slots, x3 first; one rounding at the end.
// A thread has one vector of one token's row and asks for four experts' rows
// before it adds the first.  4096 tokens of 8192 bfloat16, four choices, with x3:
// 403 MB in 68 us, 5.9 TB/s, 92 % of a plain copy's rate.
template <int TYPE, int N>
__global__ void __launch_bounds__(256) combine_kernel(CombineParams p, int tpt) {
  using E = Elem<TYPE>;
  using P = Pack<TYPE, N>;
  pdl_wait();
  pdl_trigger();
  const int64_t t = static_cast<int64_t>(blockIdx.x) * (blockDim.x / tpt) + threadIdx.x / tpt;
  if (t >= p.tokens) return;
  const int64_t nv = p.hidden / N;
  const int64_t c = static_cast<int64_t>(blockIdx.y) * tpt + threadIdx.x % tpt;
  if (c >= nv) return;
  const P* xs = static_cast<const P*>(p.x_sorted);
  float sum[N];
  if (p.x3) {
    const P a = static_cast<const P*>(p.x3)[t * nv + c];
#pragma unroll
    for (int i = 0; i < N; ++i) sum[i] = E::get(a.v[i]);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) sum[i] = 0.f;
  }
  constexpr int B = 4;  // rows in flight
  for (int j0 = 0; j0 < p.top; j0 += B) {
    P row[B];
    float w[B];
    bool has[B];
#pragma unroll
    for (int b = 0; b < B; ++b) {
      has[b] = false;
      if (j0 + b < p.top) {
        const int64_t slot = t * p.top + j0 + b;
        const int64_t pos = p.position[slot];
        has[b] = pos >= 0 && pos < p.rows;
        if (has[b]) {
          row[b] = xs[pos * nv + c];
          w[b] = p.weights ? load_scalar(p.weights, slot, p.wtype) : 1.f;
        }
      }
    }
#pragma unroll
    for (int b = 0; b < B; ++b)
      if (has[b]) {
#pragma unroll
        for (int i = 0; i < N; ++i) sum[i] = fmaf(w[b], E::get(row[b].v[i]), sum[i]);
      }
  }
  P o;
#pragma unroll
  for (int i = 0; i < N; ++i) o.v[i] = E::put(sum[i]);
  static_cast<P*>(p.out)[t * nv + c] = o;
}

// ------------------------------------------------------------------ combine's gradient
// One pass over the token's gradient and its experts' rows gives both results:
// grad_sorted[pos] = w * grad, and the dot product of grad with the row.  The
// dot products are summed per thread, over the warp by shuffles and over the
// token's warps in shared memory, always in the same order.  4096 tokens of 4096
// bfloat16, four choices: 302 MB in 50 us, 6.0 TB/s, 94 % of a plain copy's rate
// (73 us with room for eight slots' rows in every thread: half the occupancy).
// B: slots of one pass over the gradient.
template <int TYPE, int N, int B>
__global__ void __launch_bounds__(256) combine_grad_kernel(CombineGradParams p, int tpt) {
  using E = Elem<TYPE>;
  using P = Pack<TYPE, N>;
  __shared__ float part[8][B];
  pdl_wait();
  pdl_trigger();
  const int group = threadIdx.x / tpt, lane = threadIdx.x % tpt;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * (blockDim.x / tpt) + group;
  const bool live = t < p.tokens;
  const int64_t nv = p.hidden / N;
  const P* g = static_cast<const P*>(p.grad) + t * nv;
  const P* xs = static_cast<const P*>(p.x_sorted);
  P* gs = static_cast<P*>(p.grad_sorted);
  for (int j0 = 0; j0 < p.top; j0 += B) {
    float dot[B];
    int pos[B];
    float w[B];
#pragma unroll
    for (int b = 0; b < B; ++b) {
      dot[b] = 0.f;
      pos[b] = -1;
      if (live && j0 + b < p.top) {
        pos[b] = p.position[t * p.top + j0 + b];
        if (pos[b] >= p.rows) pos[b] = -1;
        w[b] = load_scalar(p.weights, t * p.top + j0 + b, p.wtype);
      }
    }
    if (live) {
      for (int64_t c = lane; c < nv; c += tpt) {
        const P gv = g[c];
        P row[B];
#pragma unroll
        for (int b = 0; b < B; ++b)
          if (pos[b] >= 0) row[b] = xs[pos[b] * nv + c];
#pragma unroll
        for (int b = 0; b < B; ++b)
          if (pos[b] >= 0) {
            P o;
#pragma unroll
            for (int i = 0; i < N; ++i) {
              const float gf = E::get(gv.v[i]);
              dot[b] = fmaf(gf, E::get(row[b].v[i]), dot[b]);
              o.v[i] = E::put(w[b] * gf);
            }
            gs[pos[b] * nv + c] = o;
          }
      }
    }
#pragma unroll
    for (int b = 0; b < B; ++b)
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) dot[b] += __shfl_xor_sync(0xffffffffu, dot[b], d);
    if (tpt > 32) {
      if ((threadIdx.x & 31) == 0)
#pragma unroll
        for (int b = 0; b < B; ++b) part[threadIdx.x >> 5][b] = dot[b];
      __syncthreads();
      if (lane < B && live && j0 + lane < p.top) {
        float v = 0.f;
        for (int w0 = 0; w0 < tpt / 32; ++w0) v += part[group * (tpt / 32) + w0][lane];
        store_scalar(p.grad_weights, t * p.top + j0 + lane, p.wtype, v);
      }
      __syncthreads();
    } else if (live) {
#pragma unroll
      for (int b = 0; b < B; ++b)
        if (lane == b && j0 + b < p.top) store_scalar(p.grad_weights, t * p.top + j0 + b, p.wtype, dot[b]);
    }
  }
}

// Threads of one row: the vectors of it, rounded up to a power of two in [lo, 256].
int threads_per_row(int64_t vecs, int lo) {
  int t = lo;
  while (t < 256 && t < vecs) t *= 2;
  return t;
}

// Largest power of two, at most `most`, that divides all of the addresses and the row's bytes.
int vector_bytes(std::initializer_list<const void*> ptrs, int64_t row_bytes, int most) {
  uintptr_t all = static_cast<uintptr_t>(row_bytes);
  for (const void* q : ptrs) all |= reinterpret_cast<uintptr_t>(q);
  int v = most;
  while (v > 1 && (all & (v - 1))) v /= 2;
  return v;
}

template <int TYPE, int N>
cudaError_t combine_as(const CombineParams& p, cudaStream_t s) {
  const int64_t nv = p.hidden / N;
  const int tpt = threads_per_row(nv, 32);
  const int per = 256 / tpt;
  const dim3 grid(static_cast<unsigned>((p.tokens + per - 1) / per), static_cast<unsigned>((nv + tpt - 1) / tpt));
  return launch_pdl(combine_kernel<TYPE, N>, grid, dim3(256), 0, 1, s, p, tpt);
}

template <int TYPE, int N, int B>
cudaError_t combine_grad_slots(const CombineGradParams& p, cudaStream_t s) {
  const int tpt = threads_per_row(p.hidden / N, 32);
  const int per = 256 / tpt;
  return launch_pdl(combine_grad_kernel<TYPE, N, B>, dim3(static_cast<unsigned>((p.tokens + per - 1) / per)),
                    dim3(256), 0, 1, s, p, tpt);
}

template <int TYPE, int N>
cudaError_t combine_grad_as(const CombineGradParams& p, cudaStream_t s) {
  return p.top <= 2   ? combine_grad_slots<TYPE, N, 2>(p, s)
         : p.top <= 4 ? combine_grad_slots<TYPE, N, 4>(p, s)
                      : combine_grad_slots<TYPE, N, 8>(p, s);
}

template <int TYPE>
cudaError_t combine_type(const CombineParams& p, cudaStream_t s) {
  constexpr int ES = sizeof(typename Elem<TYPE>::T);
  const int vb = vector_bytes({p.x_sorted, p.x3, p.out}, p.hidden * ES, 16);
  switch (vb) {
    case 16: return combine_as<TYPE, 16 / ES>(p, s);
    case 8: return combine_as<TYPE, 8 / ES>(p, s);
    case 4: return combine_as<TYPE, 4 / ES>(p, s);
    default: return combine_as<TYPE, 1>(p, s);
  }
}

template <int TYPE>
cudaError_t combine_grad_type(const CombineGradParams& p, cudaStream_t s) {
  constexpr int ES = sizeof(typename Elem<TYPE>::T);
  const int vb = vector_bytes({p.grad, p.x_sorted, p.grad_sorted}, p.hidden * ES, 16);
  switch (vb) {
    case 16: return combine_grad_as<TYPE, 16 / ES>(p, s);
    case 8: return combine_grad_as<TYPE, 8 / ES>(p, s);
    case 4: return combine_grad_as<TYPE, 4 / ES>(p, s);
    default: return combine_grad_as<TYPE, 1>(p, s);
  }
}

template <int VB, int UN>
cudaError_t dispatch_as(const DispatchParams& p, cudaStream_t s) {
  const int64_t nv = p.row_bytes / VB;
  const int tpt = threads_per_row((nv + UN - 1) / UN, 32);
  const int per = 256 / tpt;
  const dim3 grid(static_cast<unsigned>((p.tokens + per - 1) / per),
                  static_cast<unsigned>((nv + static_cast<int64_t>(tpt) * UN - 1) / (static_cast<int64_t>(tpt) * UN)));
  return launch_pdl(dispatch_kernel<VB, UN>, grid, dim3(256), 0, 1, s, p, tpt);
}

template <int VB>
cudaError_t dispatch_bytes(const DispatchParams& p, cudaStream_t s) {
  return p.tokens * (p.row_bytes / VB) >= 148 * 2048 * 4 ? dispatch_as<VB, 4>(p, s) : dispatch_as<VB, 1>(p, s);
}

size_t place_smem(int warps, int groups) { return (static_cast<size_t>(warps + 2) * (groups + 1) + 32) * 4; }

template <typename IdT>
cudaError_t sort_as(const SortParams& p, cudaStream_t s) {
  const bool cluster = p.chunks > 1 && p.chunks <= kSortCluster;
  if (p.chunks > kSortCluster) {
    const cudaError_t e = launch_pdl(sort_count_kernel<IdT>, dim3(p.chunks), dim3(256),
                                     static_cast<size_t>(p.groups + 1) * 4, 1, s, p);
    if (e != cudaSuccess) return e;
  }
  // a batch per warp where the chunk and shared memory allow it
  int threads = std::min(1024, std::max(64, (p.chunk / kBatch + 31) & ~31));
  while (place_smem(threads / 32, p.groups) > 200 * 1024) threads = (threads / 2 + 31) & ~31;
  const size_t smem = place_smem(threads / 32, p.groups);
  auto kernel = cluster ? sort_place_kernel<IdT, true> : sort_place_kernel<IdT, false>;
  if (const cudaError_t e = allow_smem(kernel, smem); e != cudaSuccess) return e;
  return launch_pdl(kernel, dim3(p.chunks), dim3(threads), smem, cluster ? p.chunks : 1, s, p);
}

}  // namespace

uint64_t plan_sort(SortParams& p) {
  // Up to 1024 slots one CTA, up to 32768 a cluster of up to eight with 1024 or
  // more each, in one launch (6162 slots: 5.0 us; with the counts in memory, two
  // launches, 6.9 us; 32768: 9.4 and 9.9); beyond, chunks of 1024 (65536: 15 us;
  // of 512: 26 us), larger ones where there would be more than 128, since every
  // CTA reads all counts.
  const int64_t slots = std::max<int64_t>(32, p.slots);
  int64_t chunk = slots;
  if (slots > 32768)
    chunk = std::max<int64_t>(1024, ((slots + 127) / 128 + 255) / 256 * 256);
  else if (slots > 1024)
    chunk = std::max<int64_t>(1024, ((slots + kSortCluster - 1) / kSortCluster + 127) / 128 * 128);
  p.chunk = static_cast<int>(chunk);
  p.chunks = static_cast<int>((slots + chunk - 1) / chunk);
  return p.chunks > kSortCluster ? static_cast<uint64_t>(p.chunks) * (p.groups + 1) * 4 : 0;
}

cudaError_t launch_sort(const SortParams& p, cudaStream_t s) {
  return p.ids64 ? sort_as<int64_t>(p, s) : sort_as<int32_t>(p, s);
}

cudaError_t launch_dispatch(const DispatchParams& p, cudaStream_t s) {
  if (p.tokens == 0 || p.rows == 0 || p.row_bytes == 0 || p.top == 0) return cudaSuccess;
  switch (vector_bytes({p.x, p.out}, p.row_bytes, 16)) {
    case 16: return dispatch_bytes<16>(p, s);
    case 8: return dispatch_bytes<8>(p, s);
    case 4: return dispatch_bytes<4>(p, s);
    case 2: return dispatch_bytes<2>(p, s);
    default: return dispatch_bytes<1>(p, s);
  }
}

cudaError_t launch_combine(const CombineParams& p, cudaStream_t s) {
  if (p.tokens == 0 || p.hidden == 0) return cudaSuccess;
  switch (p.type) {
    case kRtF16: return combine_type<kRtF16>(p, s);
    case kRtBf16: return combine_type<kRtBf16>(p, s);
    default: return combine_type<kRtF32>(p, s);
  }
}

cudaError_t launch_combine_grad(const CombineGradParams& p, cudaStream_t s) {
  if (p.tokens == 0 || p.top == 0) return cudaSuccess;
  switch (p.type) {
    case kRtF16: return combine_grad_type<kRtF16>(p, s);
    case kRtBf16: return combine_grad_type<kRtBf16>(p, s);
    default: return combine_grad_type<kRtF32>(p, s);
  }
}

}  // namespace wqmm
