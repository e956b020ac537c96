"""Token routing without a GPU: what phase 1 refuses and accepts, workspace sizes, executors, and the checks of the
torch wrappers."""
import pytest

import weight_quantized_gemm_anti_b200 as W
from weight_quantized_gemm_anti_b200 import routing

FAKE = 0x10000  # never dereferenced: phase 1 reads descriptors only
NULL, INVALID = W.ERR_PARAM_NULLPTR, W.ERR_PARAM_INVALID


@pytest.fixture(scope="module", autouse=True)
def built():
    W.build()


def T(shape, dtype, **kw):
    return W.desc(data=kw.pop("data", FAKE), dtype=dtype, shape=shape, **kw)


def call(f, *args):
    st, ws, ex = f(*args)
    if ex:
        W.wqmm_executor_destroy(ex)
    return st, ws


def sort(ids=((6, 2), W.DT_I32), groups=4, offsets=None, source=None, position=None, **kw):
    ids_d = T(*ids, **kw)
    slots = 1
    for s in ids[0]:
        slots *= s
    return call(W.route_sort_get_workspace_size, ids_d, groups, T(*(offsets or ((groups + 1,), W.DT_I32))),
                T(*(source or ((slots,), W.DT_I32))), T(*(position or (ids[0], W.DT_I32))))


def test_sort_accepts():
    assert sort() == (0, 0)
    assert sort(ids=((6,), W.DT_I64)) == (0, 0)
    assert sort(ids=((2, 3, 2), W.DT_I64), groups=2048) == (0, 0)
    assert sort(ids=((0, 2), W.DT_I32)) == (0, 0)
    st, ws = sort(ids=((5000, 8), W.DT_I32), groups=256)
    assert st == 0 and ws >= 257 * 4 * 2


@pytest.mark.parametrize("kw", [
    dict(groups=0, offsets=((1,), W.DT_I32)), dict(groups=2049), dict(ids=((6, 2), W.DT_F32)),
    dict(offsets=((4,), W.DT_I32)), dict(offsets=((5,), W.DT_I64)), dict(source=((11,), W.DT_I32)),
    dict(position=((12,), W.DT_I32)), dict(strides=(1, 6)), dict(data=FAKE + 2), dict(fmt=W.FORMAT_PACKED),
    dict(ids=((2 ** 31, 2), W.DT_I32)), dict(ids=((2 ** 30, 2), W.DT_I32)),
    dict(ids=((2 ** 31 - 1, 2 ** 31 - 1, 2 ** 31 - 1), W.DT_I32), source=((1,), W.DT_I32))])
def test_sort_refuses(kw):
    assert sort(**kw)[0] == INVALID
    assert W.wqmm_last_error()


def test_null_pointers():
    d = T((6, 2), W.DT_I32)
    assert call(W.route_sort_get_workspace_size, None, 4, d, d, d)[0] == NULL
    assert call(W.route_dispatch_get_workspace_size, None, d, d)[0] == NULL
    assert call(W.route_combine_get_workspace_size, d, None, None, None, d)[0] == NULL
    assert call(W.route_combine_grad_get_workspace_size, d, d, d, None, d, d)[0] == NULL
    assert sort(data=0)[0] == NULL


def dispatch(x=((6, 40), W.DT_BF16), position=((6, 2), W.DT_I32), out=((12, 40), None), **kw):
    return call(W.route_dispatch_get_workspace_size, T(*x, **kw), T(*position), T(out[0], out[1] or x[1]))[0]


def test_dispatch_arguments():
    for dt in (W.DT_F16, W.DT_BF16, W.DT_F32, W.DT_I8, W.DT_FP8E4M3, W.DT_I32, W.DT_I64):
        assert dispatch(x=((6, 40), dt)) == 0
    assert dispatch(x=((2, 3, 40), W.DT_F16)) == 0
    assert dispatch(out=((5, 40), None)) == 0  # fewer rows than slots: the rest is dropped
    assert dispatch(x=((0, 40), W.DT_F16), position=((0, 2), W.DT_I32)) == 0
    assert dispatch(x=((6, 1), W.DT_F32), out=((12, 1), None)) == 0
    for kw in (dict(x=((6, 40), W.DT_I4)), dict(out=((12, 41), None)), dict(out=((12, 40), W.DT_F16)),
               dict(position=((5, 2), W.DT_I32)), dict(position=((6, 2), W.DT_I64)), dict(x=((40,), W.DT_F16)),
               dict(x=((6, 0), W.DT_F16), out=((12, 0), None)), dict(out=((2, 6, 40), None)),
               dict(strides=(80, 1)), dict(data=FAKE + 1),
               dict(x=((6, 65536), W.DT_F16), out=((12, 65536), None)),
               dict(position=((6, 2 ** 31 - 1), W.DT_I32))):
        assert dispatch(**kw) == INVALID, kw


def combine(xs=((12, 40), W.DT_BF16), position=((6, 2), W.DT_I32), weights=((6, 2), W.DT_F32), x3=None,
            out=((6, 40), None), **kw):
    return call(W.route_combine_get_workspace_size, T(*xs, **kw), T(*position), None if weights is None else T(*weights),
                None if x3 is None else T(*x3), T(out[0], out[1] or xs[1]))[0]


def test_combine_arguments():
    for dt in (W.DT_F16, W.DT_BF16, W.DT_F32):
        assert combine(xs=((12, 40), dt)) == 0
        assert combine(weights=((6, 2), dt)) == 0
    assert combine(weights=None) == 0
    assert combine(x3=((6, 40), W.DT_BF16)) == 0
    assert combine(out=((2, 3, 40), None)) == 0
    assert combine(position=((6, 0), W.DT_I32), weights=((6, 0), W.DT_F32)) == 0
    for kw in (dict(xs=((12, 40), W.DT_I8)), dict(out=((6, 40), W.DT_F32)), dict(x3=((6, 40), W.DT_F32)),
               dict(x3=((7, 40), W.DT_BF16)), dict(weights=((12,), W.DT_F32)), dict(weights=((6, 2), W.DT_I32)),
               dict(position=((7, 2), W.DT_I32), weights=((7, 2), W.DT_F32)), dict(out=((6, 32), None)),
               dict(xs=((3, 4, 40), W.DT_BF16)), dict(strides=(48, 1))):
        assert combine(**kw) == INVALID, kw


def combine_grad(grad=((6, 40), W.DT_BF16), xs=None, position=((6, 2), W.DT_I32), weights=((6, 2), W.DT_F32),
                 gs=None, gw=None):
    xs = xs or ((12, 40), grad[1])
    return call(W.route_combine_grad_get_workspace_size, T(*grad), T(*xs), T(*position), T(*weights), T(*(gs or xs)),
                T(*(gw or weights)))[0]


def test_combine_grad_arguments():
    assert combine_grad() == 0
    assert combine_grad(grad=((2, 3, 40), W.DT_F32), weights=((6, 2), W.DT_F16)) == 0
    for kw in (dict(xs=((12, 40), W.DT_F16)), dict(gs=((11, 40), W.DT_BF16)), dict(gw=((6, 2), W.DT_F16)),
               dict(gw=((12,), W.DT_F32)), dict(grad=((6, 40), W.DT_I8)), dict(weights=((6, 2), W.DT_I32)),
               dict(position=((6, 3), W.DT_I32))):
        assert combine_grad(**kw) == INVALID, kw


def test_executors_are_one_shot_and_of_their_own_kind():
    d = T((6, 2), W.DT_I32)
    st, ws, ex = W.route_sort_get_workspace_size(d, 4, T((5,), W.DT_I32), T((12,), W.DT_I32), d)
    assert st == 0 and ex
    assert W.wqmm_run(0, 0, ex, 0) == W.ERR_EXECUTOR  # another operator's phase 2 refuses it and leaves it alone
    W.wqmm_executor_destroy(ex)
    assert W.route_run(0, 0, ex, 0) == W.ERR_EXECUTOR
    assert W.route_run(0, 0, None, 0) == W.ERR_EXECUTOR
    # (more slots than one cluster sorts: the counts need a workspace)
    st, ws, ex = W.route_sort_get_workspace_size(T((25000, 2), W.DT_I32), 4, T((5,), W.DT_I32), T((50000,), W.DT_I32),
                                                 T((25000, 2), W.DT_I32))
    assert st == 0 and ws > 0
    assert W.route_run(FAKE, ws - 1, ex, 0) == W.ERR_WORKSPACE  # consumed all the same
    assert W.route_run(FAKE, ws, ex, 0) == W.ERR_EXECUTOR


def test_wrappers_refuse_host_tensors():
    torch = pytest.importorskip("torch")
    ids = torch.zeros(4, 2, dtype=torch.int32)
    order = routing.TokenOrder(torch.zeros(3, dtype=torch.int32), torch.zeros(8, dtype=torch.int32), ids)
    x = torch.zeros(4, 8)
    for f in (lambda: routing.sort_tokens(ids, 2), lambda: routing.dispatch_tokens(x, order),
              lambda: routing.combine_tokens(x, order), lambda: routing.combine_tokens_grad(x, x, order, x),
              lambda: routing.expert_weight_quant_matmul(x, order, [], [])):
        with pytest.raises(ValueError, match="CUDA"):
            f()


# ------------------------------------------------------------------ memory that an output shares
# Phase 2 refuses it before it launches; the addresses are made up, so only where no GPU could be given them.
try:
    import torch
    NO_GPU = not torch.cuda.is_available()
except ImportError:
    NO_GPU = True
no_gpu = pytest.mark.skipif(not NO_GPU, reason="made-up addresses")
BIG = 1 << 20  # apart: each tensor has a megabyte of its own

TENSORS = {
    W.route_sort_get_workspace_size: dict(ids=((6, 2), W.DT_I32), offsets=((5,), W.DT_I32),
                                          source=((12,), W.DT_I32), position=((6, 2), W.DT_I32)),
    W.route_dispatch_get_workspace_size: dict(x=((6, 40), W.DT_F16), position=((6, 2), W.DT_I32),
                                              out=((12, 40), W.DT_F16)),
    W.route_combine_get_workspace_size: dict(xs=((12, 40), W.DT_F16), position=((6, 2), W.DT_I32),
                                             weights=((6, 2), W.DT_F32), x3=((6, 40), W.DT_F16),
                                             out=((6, 40), W.DT_F16)),
    W.route_combine_grad_get_workspace_size: dict(grad=((6, 40), W.DT_F16), xs=((12, 40), W.DT_F16),
                                                  position=((6, 2), W.DT_I32), weights=((6, 2), W.DT_F32),
                                                  gs=((12, 40), W.DT_F16), gw=((6, 2), W.DT_F32))}


@no_gpu
@pytest.mark.parametrize("phase1,what,at,off", [
    (f, *v) for f, cases in {
        W.route_sort_get_workspace_size: [("source", "ids", 0), ("position", "ids", 0), ("offsets", "ids", 44),
                                          ("ids", "source", 44), ("position", "source", 0)],
        W.route_dispatch_get_workspace_size: [("out", "x", 0), ("out", "x", 478), ("x", "out", 958),
                                              ("out", "position", 0)],
        W.route_combine_get_workspace_size: [("out", "xs", 0), ("out", "x3", 2), ("x3", "out", 478),
                                             ("out", "weights", 0), ("out", "position", 46)],
        W.route_combine_grad_get_workspace_size: [("gs", "grad", 0), ("gs", "xs", 2), ("gs", "weights", 0),
                                                  ("gw", "weights", 0), ("gw", "position", 0), ("gw", "xs", 0),
                                                  ("gs", "gw", 0)]}.items() for v in cases])
def test_memory_in_common_is_refused(phase1, what, at, off):
    tensors = TENSORS[phase1]
    names = list(tensors)
    address = {n: BIG * (i + 1) for i, n in enumerate(names)}
    address[what] = address[at] + off
    args = [T(*tensors[n], data=address[n]) for n in names]
    if "ids" in tensors:
        args.insert(1, 4)
    st, ws, ex = phase1(*args)
    assert st == 0, W.wqmm_last_error()
    assert W.route_run(BIG * 64, ws, ex, 0) == INVALID
    assert "shares memory" in W.wqmm_last_error()
