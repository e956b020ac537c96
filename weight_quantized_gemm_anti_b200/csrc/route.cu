// route.cu -- phase 1 and phase 2 of the token routing operators
// (include/wqmm.h, "token routing"): argument checks in the order null ->
// dtype -> attributes -> shape, and plans that launch kernels_route.cu.
#include "route.h"

#include <algorithm>

#include "host.h"

using namespace wqmm;

namespace {

constexpr int64_t kMaxSlots = 2147483647LL;
constexpr int64_t kMaxHidden = 65535;

template <typename P, cudaError_t (*LAUNCH)(const P&, cudaStream_t)>
struct RoutePlan final : OpPlan {
  P p;
  const char* what;
  RoutePlan(const P& p_, const char* what_) : p(p_), what(what_) {}
  wqmm_status run(void*, cudaStream_t s) override {
    const cudaError_t e = LAUNCH(p, s);
    return e == cudaSuccess ? WQMM_SUCCESS : cuda_fail(e, what);
  }
};

struct SortPlan final : OpPlan {
  SortParams p;
  explicit SortPlan(const SortParams& p_) : p(p_) {}
  wqmm_status run(void* workspace, cudaStream_t s) override {
    p.hist = static_cast<int*>(workspace);
    const cudaError_t e = launch_sort(p, s);
    return e == cudaSuccess ? WQMM_SUCCESS : cuda_fail(e, "token sort launch");
  }
};

int route_type(int dt) {
  switch (dt) {
    case WQMM_DT_F16: return kRtF16;
    case WQMM_DT_BF16: return kRtBf16;
    case WQMM_DT_F32: return kRtF32;
    default: return -1;
  }
}

struct Arg {
  const wqmm_tensor* t;
  const char* name;
};

// Descriptors of the tensors that are given (no product of their checked extents overflows).
wqmm_status check_args(const Arg* a, int n) {
  for (int i = 0; i < n; ++i) {
    if (!a[i].t) continue;
    const wqmm_status st = check_descriptor(a[i].t, a[i].name);
    if (st) return st;
    if (a[i].t->format != WQMM_FORMAT_ND)
      return fail(WQMM_ERR_PARAM_INVALID, "%s: only x2 of the GEMMs may use the packed format", a[i].name);
    for (int d = 0; d < a[i].t->ndim; ++d)
      if (a[i].t->shape[d] > kMaxSlots)
        return fail(WQMM_ERR_PARAM_INVALID, "%s: extent %lld is larger than 2147483647", a[i].name,
                    (long long)a[i].t->shape[d]);
  }
  return WQMM_SUCCESS;
}

// Data pointers (a tensor without elements needs none) on their element's boundary, and contiguity.
wqmm_status check_data(const Arg* a, int n) {
  for (int i = 0; i < n; ++i) {
    if (!a[i].t) continue;
    if (!contiguous(a[i].t)) return fail(WQMM_ERR_PARAM_INVALID, "%s must be contiguous", a[i].name);
    if (numel(a[i].t) == 0) continue;
    if (!a[i].t->data) return fail(WQMM_ERR_PARAM_NULLPTR, "%s: data pointer is null", a[i].name);
    const int es = dt_bytes(a[i].t->dtype);
    if (reinterpret_cast<uintptr_t>(a[i].t->data) % es)
      return fail(WQMM_ERR_PARAM_INVALID, "%s: data must be aligned to its elements (%d bytes)", a[i].name, es);
  }
  return WQMM_SUCCESS;
}

int64_t leading(const wqmm_tensor* t) {
  int64_t n = 1;
  for (int i = 0; i + 1 < t->ndim; ++i) n *= t->shape[i];
  return n;
}

// tokens and slots per token of a (T) or (..., K) tensor of slots beside rows
// of `x` ((T, H) or (b, s, H)).
wqmm_status check_slots(const wqmm_tensor* slots, const char* name, int64_t tokens, int64_t* top) {
  const int64_t t = slots->ndim == 1 ? slots->shape[0] : leading(slots);
  const int64_t k = slots->ndim == 1 ? 1 : slots->shape[slots->ndim - 1];
  if (t != tokens)
    return fail(WQMM_ERR_PARAM_INVALID, "%s must have the %lld tokens, got %lld", name, (long long)tokens, (long long)t);
  if (t > 0 && k > kMaxSlots / t)
    return fail(WQMM_ERR_PARAM_INVALID, "%s has more than %lld slots", name, (long long)kMaxSlots);
  *top = k;
  return WQMM_SUCCESS;
}

wqmm_status check_rows(const wqmm_tensor* t, const char* name) {
  if (t->ndim != 2) return fail(WQMM_ERR_PARAM_INVALID, "%s must be 2-D (rows, hidden), got %d-D", name, t->ndim);
  if (t->shape[0] > kMaxSlots) return fail(WQMM_ERR_PARAM_INVALID, "%s has more than 2147483647 rows", name);
  return WQMM_SUCCESS;
}

wqmm_status check_hidden(const wqmm_tensor* t, const char* name, int64_t hidden) {
  if (t->ndim < 2 || t->shape[t->ndim - 1] != hidden)
    return fail(WQMM_ERR_PARAM_INVALID, "%s must have the hidden size %lld as its last extent", name, (long long)hidden);
  if (hidden < 1 || hidden > kMaxHidden)
    return fail(WQMM_ERR_PARAM_INVALID, "hidden size %lld not in [1, %lld]", (long long)hidden, (long long)kMaxHidden);
  return WQMM_SUCCESS;
}

bool equal_shape(const wqmm_tensor* a, const wqmm_tensor* b) {
  if (a->ndim != b->ndim) return false;
  for (int i = 0; i < a->ndim; ++i)
    if (a->shape[i] != b->shape[i]) return false;
  return true;
}

wqmm_status no_memory() { return fail(WQMM_ERR_INNER_TILING, "out of host memory"); }

wqmm_status sort_phase1(const wqmm_tensor* ids, int64_t groups, const wqmm_tensor* offsets, const wqmm_tensor* source,
                        const wqmm_tensor* position, uint64_t* workspace_size, wqmm_executor** executor) {
  if (!ids || !offsets || !source || !position)
    return fail(WQMM_ERR_PARAM_NULLPTR, "expertIds, offsets, source and position must not be null");
  if (!workspace_size || !executor) return fail(WQMM_ERR_PARAM_NULLPTR, "workspaceSize and executor must not be null");
  *executor = nullptr;
  *workspace_size = 0;
  const Arg args[] = {{ids, "expertIds"}, {offsets, "offsets"}, {source, "source"}, {position, "position"}};
  wqmm_status st = check_args(args, 4);
  if (st) return st;
  if (ids->dtype != WQMM_DT_I32 && ids->dtype != WQMM_DT_I64)
    return fail(WQMM_ERR_PARAM_INVALID, "expertIds dtype %s not supported (int32, int64)", dt_name(ids->dtype));
  for (int i = 1; i < 4; ++i)
    if (args[i].t->dtype != WQMM_DT_I32) return fail(WQMM_ERR_PARAM_INVALID, "%s must be int32", args[i].name);
  if (groups < 1 || groups > kMaxGroups)
    return fail(WQMM_ERR_PARAM_INVALID, "numExperts %lld not in [1, %d]", (long long)groups, kMaxGroups);
  int64_t top = 0;
  st = check_slots(ids, "expertIds", ids->ndim == 1 ? ids->shape[0] : leading(ids), &top);
  if (st) return st;
  const int64_t slots = numel(ids);
  if (offsets->ndim != 1 || offsets->shape[0] != groups + 1)
    return fail(WQMM_ERR_PARAM_INVALID, "offsets must have shape (numExperts + 1) = (%lld)", (long long)groups + 1);
  if (source->ndim != 1 || source->shape[0] != slots)
    return fail(WQMM_ERR_PARAM_INVALID, "source must have shape (%lld), one entry per id", (long long)slots);
  if (!equal_shape(position, ids)) return fail(WQMM_ERR_PARAM_INVALID, "position must have the shape of expertIds");
  st = check_data(args, 4);
  if (st) return st;
  SortParams p{};
  p.ids = ids->data;
  p.ids64 = ids->dtype == WQMM_DT_I64;
  p.slots = slots;
  p.groups = static_cast<int>(groups);
  p.offsets = static_cast<int*>(offsets->data);
  p.source = static_cast<int*>(source->data);
  p.position = static_cast<int*>(position->data);
  const uint64_t ws = round_up(plan_sort(p), 256);
  auto plan = std::make_unique<SortPlan>(p);
  for (int i = 1; i < 4; ++i) plan->memories.add_out(whole(args[i].t, args[i].name));
  plan->memories.add_in(whole(ids, "expertIds"));
  return hand_out(OpKind::kRoute, std::move(plan), ws, workspace_size, executor);
}

wqmm_status dispatch_phase1(const wqmm_tensor* x, const wqmm_tensor* position, const wqmm_tensor* output,
                            uint64_t* workspace_size, wqmm_executor** executor) {
  if (!x || !position || !output) return fail(WQMM_ERR_PARAM_NULLPTR, "x, position and output must not be null");
  if (!workspace_size || !executor) return fail(WQMM_ERR_PARAM_NULLPTR, "workspaceSize and executor must not be null");
  *executor = nullptr;
  *workspace_size = 0;
  const Arg args[] = {{x, "x"}, {position, "position"}, {output, "output"}};
  wqmm_status st = check_args(args, 3);
  if (st) return st;
  const int es = dt_bytes(x->dtype);
  if (es == 0) return fail(WQMM_ERR_PARAM_INVALID, "x dtype %s cannot be dispatched", dt_name(x->dtype));
  if (output->dtype != x->dtype) return fail(WQMM_ERR_PARAM_INVALID, "output dtype must equal the x dtype");
  if (position->dtype != WQMM_DT_I32) return fail(WQMM_ERR_PARAM_INVALID, "position must be int32");
  if (x->ndim < 2) return fail(WQMM_ERR_PARAM_INVALID, "x must be 2-D (tokens, hidden) or 3-D (b, s, hidden)");
  const int64_t hidden = x->shape[x->ndim - 1], tokens = leading(x);
  st = check_hidden(x, "x", hidden);
  if (st) return st;
  if (tokens > kMaxSlots) return fail(WQMM_ERR_PARAM_INVALID, "x has more than 2147483647 tokens");
  st = check_rows(output, "output");
  if (st) return st;
  st = check_hidden(output, "output", hidden);
  if (st) return st;
  int64_t top = 0;
  st = check_slots(position, "position", tokens, &top);
  if (st) return st;
  st = check_data(args, 3);
  if (st) return st;
  DispatchParams p{};
  p.x = static_cast<const uint8_t*>(x->data);
  p.out = static_cast<uint8_t*>(output->data);
  p.position = static_cast<const int*>(position->data);
  p.tokens = tokens;
  p.rows = output->shape[0];
  p.row_bytes = hidden * es;
  p.top = static_cast<int>(top);
  auto plan = std::make_unique<RoutePlan<DispatchParams, launch_dispatch>>(p, "token dispatch launch");
  plan->memories.add_out(whole(output, "output"));
  plan->memories.add_in(whole(x, "x"));
  plan->memories.add_in(whole(position, "position"));
  return hand_out(OpKind::kRoute, std::move(plan), 0, workspace_size, executor);
}

wqmm_status combine_phase1(const wqmm_tensor* x_sorted, const wqmm_tensor* position, const wqmm_tensor* weights,
                           const wqmm_tensor* x3, const wqmm_tensor* output, uint64_t* workspace_size,
                           wqmm_executor** executor) {
  if (!x_sorted || !position || !output)
    return fail(WQMM_ERR_PARAM_NULLPTR, "xSorted, position and output must not be null");
  if (!workspace_size || !executor) return fail(WQMM_ERR_PARAM_NULLPTR, "workspaceSize and executor must not be null");
  *executor = nullptr;
  *workspace_size = 0;
  const Arg args[] = {{x_sorted, "xSorted"}, {position, "position"}, {weights, "weights"}, {x3, "x3"}, {output, "output"}};
  wqmm_status st = check_args(args, 5);
  if (st) return st;
  if (route_type(x_sorted->dtype) < 0)
    return fail(WQMM_ERR_PARAM_INVALID, "xSorted dtype %s not supported (float16, bfloat16, float32)",
                dt_name(x_sorted->dtype));
  if (output->dtype != x_sorted->dtype || (x3 && x3->dtype != x_sorted->dtype))
    return fail(WQMM_ERR_PARAM_INVALID, "output and x3 must have the xSorted dtype");
  if (position->dtype != WQMM_DT_I32) return fail(WQMM_ERR_PARAM_INVALID, "position must be int32");
  if (weights && route_type(weights->dtype) < 0)
    return fail(WQMM_ERR_PARAM_INVALID, "weights dtype %s not supported (float16, bfloat16, float32)",
                dt_name(weights->dtype));
  st = check_rows(x_sorted, "xSorted");
  if (st) return st;
  const int64_t hidden = x_sorted->shape[1];
  st = check_hidden(output, "output", hidden);
  if (st) return st;
  const int64_t tokens = leading(output);
  if (tokens > kMaxSlots) return fail(WQMM_ERR_PARAM_INVALID, "output has more than 2147483647 tokens");
  if (x3 && !equal_shape(x3, output)) return fail(WQMM_ERR_PARAM_INVALID, "x3 must have the output shape");
  int64_t top = 0;
  st = check_slots(position, "position", tokens, &top);
  if (st) return st;
  if (weights && !equal_shape(weights, position))
    return fail(WQMM_ERR_PARAM_INVALID, "weights must have the shape of position");
  st = check_data(args, 5);
  if (st) return st;
  CombineParams p{};
  p.x_sorted = x_sorted->data;
  p.position = static_cast<const int*>(position->data);
  p.weights = weights ? weights->data : nullptr;
  p.x3 = x3 ? x3->data : nullptr;
  p.out = output->data;
  p.tokens = tokens;
  p.rows = x_sorted->shape[0];
  p.hidden = hidden;
  p.top = static_cast<int>(top);
  p.type = route_type(x_sorted->dtype);
  p.wtype = weights ? route_type(weights->dtype) : kRtF32;
  auto plan = std::make_unique<RoutePlan<CombineParams, launch_combine>>(p, "token combine launch");
  plan->memories.add_out(whole(output, "output"));
  plan->memories.add_in(whole(x_sorted, "xSorted"));
  plan->memories.add_in(whole(position, "position"));
  if (weights) plan->memories.add_in(whole(weights, "weights"));
  if (x3) plan->memories.add_in(whole(x3, "x3", 0));
  return hand_out(OpKind::kRoute, std::move(plan), 0, workspace_size, executor);
}

wqmm_status combine_grad_phase1(const wqmm_tensor* grad, const wqmm_tensor* x_sorted, const wqmm_tensor* position,
                                const wqmm_tensor* weights, const wqmm_tensor* grad_sorted,
                                const wqmm_tensor* grad_weights, uint64_t* workspace_size, wqmm_executor** executor) {
  if (!grad || !x_sorted || !position || !weights || !grad_sorted || !grad_weights)
    return fail(WQMM_ERR_PARAM_NULLPTR,
                "grad, xSorted, position, weights, gradSorted and gradWeights must not be null");
  if (!workspace_size || !executor) return fail(WQMM_ERR_PARAM_NULLPTR, "workspaceSize and executor must not be null");
  *executor = nullptr;
  *workspace_size = 0;
  const Arg args[] = {{grad, "grad"},       {x_sorted, "xSorted"},      {position, "position"},
                      {weights, "weights"}, {grad_sorted, "gradSorted"}, {grad_weights, "gradWeights"}};
  wqmm_status st = check_args(args, 6);
  if (st) return st;
  if (route_type(grad->dtype) < 0)
    return fail(WQMM_ERR_PARAM_INVALID, "grad dtype %s not supported (float16, bfloat16, float32)",
                dt_name(grad->dtype));
  if (x_sorted->dtype != grad->dtype || grad_sorted->dtype != grad->dtype)
    return fail(WQMM_ERR_PARAM_INVALID, "xSorted and gradSorted must have the grad dtype");
  if (position->dtype != WQMM_DT_I32) return fail(WQMM_ERR_PARAM_INVALID, "position must be int32");
  if (route_type(weights->dtype) < 0)
    return fail(WQMM_ERR_PARAM_INVALID, "weights dtype %s not supported (float16, bfloat16, float32)",
                dt_name(weights->dtype));
  if (grad_weights->dtype != weights->dtype)
    return fail(WQMM_ERR_PARAM_INVALID, "gradWeights must have the weights dtype");
  st = check_rows(x_sorted, "xSorted");
  if (st) return st;
  const int64_t hidden = x_sorted->shape[1];
  st = check_hidden(grad, "grad", hidden);
  if (st) return st;
  if (!equal_shape(grad_sorted, x_sorted))
    return fail(WQMM_ERR_PARAM_INVALID, "gradSorted must have the shape of xSorted");
  const int64_t tokens = leading(grad);
  if (tokens > kMaxSlots) return fail(WQMM_ERR_PARAM_INVALID, "grad has more than 2147483647 tokens");
  int64_t top = 0;
  st = check_slots(position, "position", tokens, &top);
  if (st) return st;
  if (!equal_shape(weights, position) || !equal_shape(grad_weights, position))
    return fail(WQMM_ERR_PARAM_INVALID, "weights and gradWeights must have the shape of position");
  st = check_data(args, 6);
  if (st) return st;
  CombineGradParams p{};
  p.grad = grad->data;
  p.x_sorted = x_sorted->data;
  p.position = static_cast<const int*>(position->data);
  p.weights = weights->data;
  p.grad_sorted = grad_sorted->data;
  p.grad_weights = grad_weights->data;
  p.tokens = tokens;
  p.rows = x_sorted->shape[0];
  p.hidden = hidden;
  p.top = static_cast<int>(top);
  p.type = route_type(grad->dtype);
  p.wtype = route_type(weights->dtype);
  auto plan =
      std::make_unique<RoutePlan<CombineGradParams, launch_combine_grad>>(p, "token combine gradient launch");
  plan->memories.add_out(whole(grad_sorted, "gradSorted"));
  plan->memories.add_out(whole(grad_weights, "gradWeights"));
  plan->memories.add_in(whole(grad, "grad"));
  plan->memories.add_in(whole(x_sorted, "xSorted", 0));
  plan->memories.add_in(whole(position, "position"));
  plan->memories.add_in(whole(weights, "weights"));
  return hand_out(OpKind::kRoute, std::move(plan), 0, workspace_size, executor);
}

}  // namespace

// The only exception below is an allocation that fails: it ends here, not in the caller's C code.
extern "C" wqmm_status route_sort_get_workspace_size(const wqmm_tensor* expert_ids, int64_t num_experts,
                                                     const wqmm_tensor* offsets, const wqmm_tensor* source,
                                                     const wqmm_tensor* position, uint64_t* workspace_size,
                                                     wqmm_executor** executor) try {
  return sort_phase1(expert_ids, num_experts, offsets, source, position, workspace_size, executor);
} catch (...) {
  return no_memory();
}

extern "C" wqmm_status route_dispatch_get_workspace_size(const wqmm_tensor* x, const wqmm_tensor* position,
                                                         const wqmm_tensor* output, uint64_t* workspace_size,
                                                         wqmm_executor** executor) try {
  return dispatch_phase1(x, position, output, workspace_size, executor);
} catch (...) {
  return no_memory();
}

extern "C" wqmm_status route_combine_get_workspace_size(const wqmm_tensor* x_sorted, const wqmm_tensor* position,
                                                        const wqmm_tensor* weights, const wqmm_tensor* x3,
                                                        const wqmm_tensor* output, uint64_t* workspace_size,
                                                        wqmm_executor** executor) try {
  return combine_phase1(x_sorted, position, weights, x3, output, workspace_size, executor);
} catch (...) {
  return no_memory();
}

extern "C" wqmm_status route_combine_grad_get_workspace_size(const wqmm_tensor* grad, const wqmm_tensor* x_sorted,
                                                             const wqmm_tensor* position, const wqmm_tensor* weights,
                                                             const wqmm_tensor* grad_sorted,
                                                             const wqmm_tensor* grad_weights,
                                                             uint64_t* workspace_size, wqmm_executor** executor) try {
  return combine_grad_phase1(grad, x_sorted, position, weights, grad_sorted, grad_weights, workspace_size, executor);
} catch (...) {
  return no_memory();
}

extern "C" wqmm_status route_run(void* workspace, uint64_t workspace_size, wqmm_executor* executor,
                                 wqmm_stream stream) try {
  return run_plan(OpKind::kRoute, workspace, workspace_size, executor, stream);
} catch (...) {
  return no_memory();
}
