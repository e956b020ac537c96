// lora.cu -- phase 1 and phase 2 of the low-rank adapter operators
// (include/wqmm.h, "low-rank adapters"): argument checks in the order null ->
// dtype -> attributes -> shape, and plans that launch lora_few.cu, lora_shrink.cu, lora_expand.cu
// and lora_outer.cu.
#include "lora.h"

#include "host.h"
#include "route.h"

using namespace wqmm;

namespace {

constexpr int64_t kMaxRank = 128;
// Row numbers and the next tile's stay within 32 bits.
constexpr int64_t kMaxRows = 1 << 26;
// In the weights' gradients one CTA may have all rows of an adapter (few items of many adapters), and the warps that
// write its sums wait for it, two seconds at most.  A step of 64 rows copies 48 KB at the largest rank: 2^22 rows of
// float16 at rank 128 (all of one of 100 adapters, k = n = 32) take 90 ms, so these 0.36 s, a fifth of the limit.
constexpr int64_t kMaxGradRows = 1 << 24;

struct Arg {
  const wqmm_tensor* t;
  const char* name;
};

wqmm_status check_args(const Arg* a, int n) {
  for (int i = 0; i < n; ++i) {
    if (!a[i].t) continue;
    const wqmm_status st = check_descriptor(a[i].t, a[i].name);
    if (st) return st;
    if (a[i].t->format != WQMM_FORMAT_ND)
      return fail(WQMM_ERR_PARAM_INVALID, "%s: only x2 of the GEMMs may use the packed format", a[i].name);
    for (int d = 0; d < a[i].t->ndim; ++d)
      if (a[i].t->shape[d] > 2147483647LL)
        return fail(WQMM_ERR_PARAM_INVALID, "%s: extent %lld is larger than 2147483647", a[i].name,
                    (long long)a[i].t->shape[d]);
  }
  return WQMM_SUCCESS;
}

wqmm_status check_pointer(const wqmm_tensor* t, const char* name, int align) {
  if (!t->data) return fail(WQMM_ERR_PARAM_NULLPTR, "%s: data pointer is null", name);
  if (reinterpret_cast<uintptr_t>(t->data) % align)
    return fail(WQMM_ERR_PARAM_INVALID, "%s: data must be %d-byte aligned", name, align);
  return WQMM_SUCCESS;
}

// Rows of `len` elements, (m, len) or (b, s, len): neighbours within a row, the
// rows at one stride of a multiple of 8 elements.
wqmm_status check_matrix(const wqmm_tensor* t, const char* name, int64_t* m, int64_t* len, int64_t* ld) {
  if (t->ndim != 2 && t->ndim != 3)
    return fail(WQMM_ERR_PARAM_INVALID, "%s must be 2-D (m, len) or 3-D (b, s, len), got %d-D", name, t->ndim);
  const int last = t->ndim - 1;
  *len = t->shape[last];
  *m = t->ndim == 2 ? t->shape[0] : t->shape[0] * t->shape[1];
  if (*m < 1 || *m > kMaxRows)
    return fail(WQMM_ERR_PARAM_INVALID, "%s: %lld rows, not in [1, %lld]", name, (long long)*m, (long long)kMaxRows);
  if (*len < 1 || *len > 65535 || *len % 32 != 0)
    return fail(WQMM_ERR_PARAM_INVALID, "%s: row length %lld must be a multiple of 32 in [32, 65535]", name,
                (long long)*len);
  if (t->strides[last] != 1) return fail(WQMM_ERR_PARAM_INVALID, "%s: the elements of a row must be neighbours", name);
  *ld = *len;
  if (*m > 1) {
    if (t->ndim == 2) {
      *ld = t->strides[0];
    } else if (t->shape[1] == 1) {
      *ld = t->strides[0];
    } else {
      *ld = t->strides[1];
      if (t->shape[0] > 1 && (t->strides[0] / t->shape[1] != *ld || t->strides[0] % t->shape[1] != 0))
        return fail(WQMM_ERR_PARAM_INVALID, "%s: all rows must be at one stride", name);
    }
  }
  if (*ld < *len || *ld % 8 != 0 || *ld > (int64_t{1} << 31))
    return fail(WQMM_ERR_PARAM_INVALID,
                "%s: the row stride %lld must be a multiple of 8, at least the row's length and at most 2^31", name,
                (long long)*ld);
  return check_pointer(t, name, 16);
}

// What lora and lora_grad have in common.
struct Problem {
  LoraRows rows;
  const uint16_t* a;
  const uint16_t* b;
  const float* scale;
  LoraMat x;
  int k, n, rank;
  bool bf16;
};

wqmm_status check_problem(const wqmm_tensor* x1, const wqmm_tensor* a, const wqmm_tensor* b, const wqmm_tensor* scale,
                          const wqmm_tensor* offsets, const wqmm_tensor* source, Problem* out) {
  int64_t m = 0, k = 0, ld = 0;
  wqmm_status st = check_matrix(x1, "x1", &m, &k, &ld);
  if (st) return st;
  if (a->ndim != 3 || b->ndim != 3)
    return fail(WQMM_ERR_PARAM_INVALID, "loraA must be 3-D (adapters, rank, k), loraB 3-D (adapters, n, rank)");
  const int64_t adapters = a->shape[0], rank = a->shape[1], n = b->shape[1];
  if (adapters < 1 || adapters > kMaxGroups)
    return fail(WQMM_ERR_PARAM_INVALID, "%lld adapters, not in [1, %d]", (long long)adapters, kMaxGroups);
  if (rank < 8 || rank > kMaxRank || rank % 8 != 0)
    return fail(WQMM_ERR_PARAM_INVALID, "rank %lld must be a multiple of 8 in [8, %lld]", (long long)rank,
                (long long)kMaxRank);
  if (a->shape[2] != k) return fail(WQMM_ERR_PARAM_INVALID, "k of x1 and loraA must be equal");
  if (b->shape[0] != adapters || b->shape[2] != rank)
    return fail(WQMM_ERR_PARAM_INVALID, "loraB must have shape (adapters, n, rank) = (%lld, n, %lld)",
                (long long)adapters, (long long)rank);
  if (n < 32 || n > 65535 || n % 32 != 0)
    return fail(WQMM_ERR_PARAM_INVALID, "n = %lld must be a multiple of 32 in [32, 65535]", (long long)n);
  if (!contiguous(a) || !contiguous(b)) return fail(WQMM_ERR_PARAM_INVALID, "loraA and loraB must be contiguous");
  if (scale && (scale->ndim != 1 || scale->shape[0] != adapters || !contiguous(scale)))
    return fail(WQMM_ERR_PARAM_INVALID, "scale must be contiguous with shape (adapters) = (%lld)", (long long)adapters);
  if (offsets->ndim != 1 || offsets->shape[0] != adapters + 1 || !contiguous(offsets))
    return fail(WQMM_ERR_PARAM_INVALID, "offsets must be contiguous with shape (adapters + 1) = (%lld)",
                (long long)adapters + 1);
  if (source->ndim != 1 || source->shape[0] != m || !contiguous(source))
    return fail(WQMM_ERR_PARAM_INVALID, "source must be contiguous with shape (m) = (%lld)", (long long)m);
  if ((st = check_pointer(a, "loraA", 16))) return st;
  if ((st = check_pointer(b, "loraB", 16))) return st;
  if (scale && (st = check_pointer(scale, "scale", 4))) return st;
  if ((st = check_pointer(offsets, "offsets", 4))) return st;
  if ((st = check_pointer(source, "source", 4))) return st;
  out->rows = {static_cast<const int*>(offsets->data), static_cast<const int*>(source->data),
               static_cast<int>(adapters), m};
  out->a = static_cast<const uint16_t*>(a->data);
  out->b = static_cast<const uint16_t*>(b->data);
  out->scale = scale ? static_cast<const float*>(scale->data) : nullptr;
  out->x = {static_cast<const uint16_t*>(x1->data), ld};
  out->k = static_cast<int>(k);
  out->n = static_cast<int>(n);
  out->rank = static_cast<int>(rank);
  out->bf16 = x1->dtype == WQMM_DT_BF16;
  return WQMM_SUCCESS;
}

wqmm_status check_dtypes(const wqmm_tensor* x1, const Arg* same, int n, const wqmm_tensor* scale,
                         const wqmm_tensor* offsets, const wqmm_tensor* source) {
  if (x1->dtype != WQMM_DT_F16 && x1->dtype != WQMM_DT_BF16)
    return fail(WQMM_ERR_PARAM_INVALID, "x1 dtype %s not supported (float16, bfloat16)", dt_name(x1->dtype));
  for (int i = 0; i < n; ++i)
    if (same[i].t && same[i].t->dtype != x1->dtype)
      return fail(WQMM_ERR_PARAM_INVALID, "%s dtype %s must equal the x1 dtype %s", same[i].name,
                  dt_name(same[i].t->dtype), dt_name(x1->dtype));
  if (scale && scale->dtype != WQMM_DT_F32) return fail(WQMM_ERR_PARAM_INVALID, "scale must be float32");
  if (offsets->dtype != WQMM_DT_I32 || source->dtype != WQMM_DT_I32)
    return fail(WQMM_ERR_PARAM_INVALID, "offsets and source must be int32");
  return WQMM_SUCCESS;
}

// A matrix of `m` rows of `len`, named by the caller.
wqmm_status check_like(const wqmm_tensor* t, const char* name, int64_t m, int64_t len, int64_t* ld) {
  int64_t tm = 0, tl = 0;
  const wqmm_status st = check_matrix(t, name, &tm, &tl, ld);
  if (st) return st;
  if (tm != m || tl != len)
    return fail(WQMM_ERR_PARAM_INVALID, "%s must have %lld rows of %lld", name, (long long)m, (long long)len);
  return WQMM_SUCCESS;
}

// An addend and a result: the same tensor (in place) or two that do not start together.
wqmm_status check_in_place(const wqmm_tensor* in, int64_t ld_in, const wqmm_tensor* out, int64_t ld_out,
                           const char* name) {
  if (in && in->data == out->data && ld_in != ld_out)
    return fail(WQMM_ERR_PARAM_INVALID, "%s in place must have the result's row stride", name);
  return WQMM_SUCCESS;
}

// The memory of rows of 16-bit numbers.
Memory rows_of(const void* p, const char* name, int64_t m, int64_t len, int64_t ld, int may_be = -1) {
  return {name, p, m, 2 * len, 2 * ld, may_be};
}

void add_weights(Memories& to, const wqmm_tensor* a, const wqmm_tensor* b, const wqmm_tensor* scale,
                 const wqmm_tensor* offsets, const wqmm_tensor* source) {
  to.add_in(whole(a, "loraA"));
  to.add_in(whole(b, "loraB"));
  if (scale) to.add_in(whole(scale, "scale"));
  to.add_in(whole(offsets, "offsets"));
  to.add_in(whole(source, "source"));
}

uint64_t low_bytes(const Problem& p) {
  return round_up(static_cast<uint64_t>(p.rows.m) * 2 * lora_padded_rank(p.rank) * 2, 256) +
         round_up(static_cast<uint64_t>(p.rows.m) * 4, 256);
}

LoraLow low_at(const Problem& p, uint8_t* at) {
  return {reinterpret_cast<uint16_t*>(at),
          reinterpret_cast<float*>(at + round_up(static_cast<uint64_t>(p.rows.m) * 2 * lora_padded_rank(p.rank) * 2, 256))};
}

struct AddPlan final : OpPlan {
  Problem p;
  LoraMat y;
  uint16_t* out;
  int64_t ldo;
  bool few;  // one launch without a workspace
  wqmm_status run(void* workspace, cudaStream_t s) override {
    const LoraLow low = few ? LoraLow{} : low_at(p, static_cast<uint8_t*>(workspace));
    const ShrinkParams sp[1] = {{p.x, p.a, p.scale, low, p.k}};
    const ExpandParams ep{low, p.b, y, out, ldo, p.n, y.p != out};
    cudaError_t e;
    if (few) {
      e = launch_lora_few(p.rows, sp[0], ep, p.rank, p.bf16, sm_count(), s);
      return e == cudaSuccess ? WQMM_SUCCESS : cuda_fail(e, "adapter launch");
    }
    e = launch_lora_shrink(p.rows, sp, 1, p.rank, p.bf16, sm_count(), s);
    if (e != cudaSuccess) return cuda_fail(e, "adapter contraction launch");
    e = launch_lora_expand(p.rows, ep, p.rank, false, p.bf16, sm_count(), s);
    return e == cudaSuccess ? WQMM_SUCCESS : cuda_fail(e, "adapter expansion launch");
  }
};

struct GradPlan final : OpPlan {
  Problem p;
  LoraMat grad, gx_in;
  uint16_t* gx;
  int64_t ldgx;
  uint16_t* ga;
  uint16_t* gb;
  // Whether `in`, rows of `len`, reaches into the memory between grad_x's first row and its last.
  bool shares(const LoraMat& in, int64_t len) const {
    const int64_t last = p.rows.m - 1;
    return gx && in.p < gx + last * ldgx + p.k && gx < in.p + last * in.ld + len;
  }
  cudaError_t input(const LoraLow& back, cudaStream_t s) const {
    if (!gx) return cudaSuccess;
    const ExpandParams ep{back, p.a, gx_in, gx, ldgx, p.k, gx_in.p != gx};
    return launch_lora_expand(p.rows, ep, p.rank, true, p.bf16, sm_count(), s);
  }
  wqmm_status run(void* workspace, cudaStream_t s) override {
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    const LoraLow low = low_at(p, ws), back = low_at(p, ws + low_bytes(p));
    const ShrinkParams sp[2] = {{p.x, p.a, p.scale, low, p.k}, {grad, p.b, p.scale, back, p.n}};
    cudaError_t e = launch_lora_shrink(p.rows, sp, 2, p.rank, p.bf16, sm_count(), s);
    if (e != cudaSuccess) return cuda_fail(e, "adapter contraction launch");
    // The weights' gradients read x1 and grad again, the input's only back: with many rows the former go first,
    // while x1 and grad are in the L2 cache (4096 x 4096 x 4096: 58 and 62 us); with few the latter, since the
    // former's CTAs can begin beside its last ones (64 rows, 32 adapters: 22 and 29 us).
    // A grad_x that is x1 or grad itself is written last.
    const bool input_first = lora_few_rows(p.rows, p.rank) && !shares(p.x, p.k) && !shares(grad, p.n);
    if (input_first && (e = input(back, s)) != cudaSuccess) return cuda_fail(e, "adapter input gradient launch");
    const OuterParams op[2] = {{p.x, back, ga, p.k, 1}, {grad, low, gb, p.n, 0}};
    e = launch_lora_outer(p.rows, op, p.rank, p.bf16, sm_count(), s);
    if (e != cudaSuccess) return cuda_fail(e, "adapter weight gradient launch");
    if (!input_first && (e = input(back, s)) != cudaSuccess) return cuda_fail(e, "adapter input gradient launch");
    return WQMM_SUCCESS;
  }
};

wqmm_status add_phase1(const wqmm_tensor* x1, const wqmm_tensor* a, const wqmm_tensor* b, const wqmm_tensor* scale,
                       const wqmm_tensor* offsets, const wqmm_tensor* source, const wqmm_tensor* y,
                       const wqmm_tensor* output, uint64_t* workspace_size, wqmm_executor** executor) {
  if (!x1 || !a || !b || !offsets || !source || !output)
    return fail(WQMM_ERR_PARAM_NULLPTR, "x1, loraA, loraB, offsets, source and output must not be null");
  if (!workspace_size || !executor) return fail(WQMM_ERR_PARAM_NULLPTR, "workspaceSize and executor must not be null");
  *executor = nullptr;
  *workspace_size = 0;
  const Arg args[] = {{x1, "x1"},           {a, "loraA"},       {b, "loraB"}, {y, "y"}, {output, "output"},
                      {scale, "scale"}, {offsets, "offsets"}, {source, "source"}};
  wqmm_status st = check_args(args, 8);
  if (st) return st;
  if ((st = check_dtypes(x1, args + 1, 4, scale, offsets, source))) return st;
  auto plan = std::make_unique<AddPlan>();
  if ((st = check_problem(x1, a, b, scale, offsets, source, &plan->p))) return st;
  const Problem& p = plan->p;
  if ((st = check_like(output, "output", p.rows.m, p.n, &plan->ldo))) return st;
  plan->out = static_cast<uint16_t*>(output->data);
  plan->y = {nullptr, 0};
  if (y) {
    if ((st = check_like(y, "y", p.rows.m, p.n, &plan->y.ld))) return st;
    if ((st = check_in_place(y, plan->y.ld, output, plan->ldo, "y"))) return st;
    plan->y.p = static_cast<const uint16_t*>(y->data);
  }
  plan->memories.add_out(rows_of(output->data, "output", p.rows.m, p.n, plan->ldo));
  plan->memories.add_in(rows_of(p.x.p, "x1", p.rows.m, p.k, p.x.ld, 0));
  if (y) plan->memories.add_in(rows_of(y->data, "y", p.rows.m, p.n, plan->y.ld, 0));
  add_weights(plan->memories, a, b, scale, offsets, source);
  plan->few = lora_one_launch(p.rows, p.rank, plan->y.p != plan->out, sm_count());
  const uint64_t workspace = plan->few ? 0 : low_bytes(p);
  return hand_out(OpKind::kLora, std::move(plan), workspace, workspace_size, executor);
}

wqmm_status grad_phase1(const wqmm_tensor* grad, const wqmm_tensor* x1, const wqmm_tensor* a, const wqmm_tensor* b,
                        const wqmm_tensor* scale, const wqmm_tensor* offsets, const wqmm_tensor* source,
                        const wqmm_tensor* gx_in, const wqmm_tensor* gx, const wqmm_tensor* ga, const wqmm_tensor* gb,
                        uint64_t* workspace_size, wqmm_executor** executor) {
  if (!grad || !x1 || !a || !b || !offsets || !source || !ga || !gb)
    return fail(WQMM_ERR_PARAM_NULLPTR,
                "grad, x1, loraA, loraB, offsets, source, gradA and gradB must not be null");
  if (gx_in && !gx) return fail(WQMM_ERR_PARAM_NULLPTR, "gradX must not be null beside an addend gradXIn");
  if (!workspace_size || !executor) return fail(WQMM_ERR_PARAM_NULLPTR, "workspaceSize and executor must not be null");
  *executor = nullptr;
  *workspace_size = 0;
  const Arg args[] = {{x1, "x1"},       {grad, "grad"}, {a, "loraA"},  {b, "loraB"},         {gx_in, "gradXIn"},
                      {gx, "gradX"}, {ga, "gradA"}, {gb, "gradB"}, {scale, "scale"}, {offsets, "offsets"}, {source, "source"}};
  wqmm_status st = check_args(args, 11);
  if (st) return st;
  if ((st = check_dtypes(x1, args + 1, 7, scale, offsets, source))) return st;
  auto plan = std::make_unique<GradPlan>();
  if ((st = check_problem(x1, a, b, scale, offsets, source, &plan->p))) return st;
  const Problem& p = plan->p;
  if (p.rows.m > kMaxGradRows)
    return fail(WQMM_ERR_PARAM_INVALID, "x1: %lld rows, the gradients take at most %lld", (long long)p.rows.m,
                (long long)kMaxGradRows);
  if ((st = check_like(grad, "grad", p.rows.m, p.n, &plan->grad.ld))) return st;
  plan->grad.p = static_cast<const uint16_t*>(grad->data);
  plan->gx = nullptr;
  plan->gx_in = {nullptr, 0};
  plan->ldgx = 0;
  if (gx) {
    if ((st = check_like(gx, "gradX", p.rows.m, p.k, &plan->ldgx))) return st;
    plan->gx = static_cast<uint16_t*>(gx->data);
  }
  if (gx_in) {
    if ((st = check_like(gx_in, "gradXIn", p.rows.m, p.k, &plan->gx_in.ld))) return st;
    if ((st = check_in_place(gx_in, plan->gx_in.ld, gx, plan->ldgx, "gradXIn"))) return st;
    plan->gx_in.p = static_cast<const uint16_t*>(gx_in->data);
  }
  const wqmm_tensor* like[] = {a, b};
  const wqmm_tensor* of[] = {ga, gb};
  const char* names[] = {"gradA", "gradB"};
  for (int i = 0; i < 2; ++i) {
    bool same = of[i]->ndim == 3;
    for (int d = 0; same && d < 3; ++d) same = of[i]->shape[d] == like[i]->shape[d];
    if (!same || !contiguous(of[i]))
      return fail(WQMM_ERR_PARAM_INVALID, "%s must be contiguous with its adapter's shape", names[i]);
    if ((st = check_pointer(of[i], names[i], 16))) return st;
  }
  plan->ga = static_cast<uint16_t*>(ga->data);
  plan->gb = static_cast<uint16_t*>(gb->data);
  if (gx) plan->memories.add_out(rows_of(gx->data, "gradX", p.rows.m, p.k, plan->ldgx));
  plan->memories.add_out(whole(ga, "gradA"));
  plan->memories.add_out(whole(gb, "gradB"));
  const int first = gx ? 0 : -1;
  plan->memories.add_in(rows_of(p.x.p, "x1", p.rows.m, p.k, p.x.ld, first));
  plan->memories.add_in(rows_of(grad->data, "grad", p.rows.m, p.n, plan->grad.ld, first));
  if (gx_in) plan->memories.add_in(rows_of(gx_in->data, "gradXIn", p.rows.m, p.k, plan->gx_in.ld, first));
  add_weights(plan->memories, a, b, scale, offsets, source);
  return hand_out(OpKind::kLora, std::move(plan), 2 * low_bytes(p), workspace_size, executor);
}

wqmm_status no_memory() { return fail(WQMM_ERR_INNER_TILING, "out of host memory"); }

}  // namespace

// The only exception below is an allocation that fails: it ends here, not in the caller's C code.
extern "C" wqmm_status lora_get_workspace_size(const wqmm_tensor* x1, const wqmm_tensor* lora_a,
                                               const wqmm_tensor* lora_b, const wqmm_tensor* scale,
                                               const wqmm_tensor* offsets, const wqmm_tensor* source,
                                               const wqmm_tensor* y, const wqmm_tensor* output,
                                               uint64_t* workspace_size, wqmm_executor** executor) try {
  return add_phase1(x1, lora_a, lora_b, scale, offsets, source, y, output, workspace_size, executor);
} catch (...) {
  return no_memory();
}

extern "C" wqmm_status lora_grad_get_workspace_size(const wqmm_tensor* grad, const wqmm_tensor* x1,
                                                    const wqmm_tensor* lora_a, const wqmm_tensor* lora_b,
                                                    const wqmm_tensor* scale, const wqmm_tensor* offsets,
                                                    const wqmm_tensor* source, const wqmm_tensor* grad_x_in,
                                                    const wqmm_tensor* grad_x, const wqmm_tensor* grad_a,
                                                    const wqmm_tensor* grad_b, uint64_t* workspace_size,
                                                    wqmm_executor** executor) try {
  return grad_phase1(grad, x1, lora_a, lora_b, scale, offsets, source, grad_x_in, grad_x, grad_a, grad_b,
                     workspace_size, executor);
} catch (...) {
  return no_memory();
}

extern "C" wqmm_status lora_run(void* workspace, uint64_t workspace_size, wqmm_executor* executor,
                                wqmm_stream stream) try {
  return run_plan(OpKind::kLora, workspace, workspace_size, executor, stream);
} catch (...) {
  return no_memory();
}
