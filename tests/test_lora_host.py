"""Low-rank adapters without a GPU: what phase 1 refuses and accepts, workspace sizes, executors, and the checks of the
torch wrappers."""
import pytest

import weight_quantized_gemm_anti_b200 as W
from weight_quantized_gemm_anti_b200 import lora
from weight_quantized_gemm_anti_b200.routing import TokenOrder

FAKE = 0x10000  # never dereferenced: phase 1 reads descriptors only
NULL, INVALID = W.ERR_PARAM_NULLPTR, W.ERR_PARAM_INVALID
F16, BF16, F32, I32 = W.DT_F16, W.DT_BF16, W.DT_F32, W.DT_I32


@pytest.fixture(scope="module", autouse=True)
def built():
    W.build()


def T(shape, dtype, strides=None, data=FAKE, fmt=W.FORMAT_ND):
    return W.desc(data=data, dtype=dtype, shape=shape, strides=strides, fmt=fmt)


def call(f, *args):
    st, ws, ex = f(*(None if a is None else T(*a[:2], **(a[2] if len(a) > 2 else {})) for a in args))
    if ex:
        W.wqmm_executor_destroy(ex)
    return st, ws


ADD = dict(x1=((6, 64), BF16), a=((3, 16, 64), BF16), b=((3, 96, 16), BF16), scale=((3,), F32), offsets=((4,), I32),
           source=((6,), I32), y=((6, 96), BF16), out=((6, 96), BF16))


def add(**kw):
    t = {**ADD, **kw}
    return call(W.lora_get_workspace_size, t["x1"], t["a"], t["b"], t["scale"], t["offsets"], t["source"], t["y"],
                t["out"])


def test_add_accepts():
    assert add() == (0, 0)  # one launch, no workspace
    many = dict(x1=((5000, 64), BF16), a=((3, 32, 64), BF16), b=((3, 96, 32), BF16), source=((5000,), I32),
                y=((5000, 96), BF16), out=((5000, 96), BF16))
    st, ws = add(**many)
    assert st == 0 and ws >= 5000 * 2 * 32 * 2
    assert add(y=None)[0] == 0 and add(scale=None)[0] == 0
    assert add(x1=((2, 3, 64), BF16), y=((2, 3, 96), BF16), out=((6, 96), BF16))[0] == 0
    # slices of wider matrices; three dimensions whose rows are at one stride
    assert add(x1=((6, 64), BF16, dict(strides=(200, 1))), y=None,
               out=((6, 96), BF16, dict(strides=(288, 1))))[0] == 0
    assert add(x1=((2, 3, 64), BF16, dict(strides=(600, 200, 1))))[0] == 0
    assert add(x1=((6, 1, 64), BF16, dict(strides=(72, 1, 1))))[0] == 0
    assert add(x1=((1, 6, 64), BF16, dict(strides=(8, 72, 1))))[0] == 0
    for rank in (8, 24, 128):
        assert add(a=((3, rank, 64), BF16), b=((3, 96, rank), BF16))[0] == 0
    one = dict(x1=((1, 64), F16, dict(strides=(3, 1))), a=((3, 16, 64), F16), b=((3, 96, 16), F16), source=((1,), I32),
               y=None, out=((1, 96), F16))
    assert add(**one)[0] == 0  # a single row has no stride


@pytest.mark.parametrize("kw", [
    dict(x1=((6, 64), F32)), dict(x1=((6, 64), F16)), dict(x1=((0, 64), BF16)), dict(x1=((64,), BF16)),
    dict(x1=((6, 48), BF16), a=((3, 16, 48), BF16)), dict(x1=((6, 64), BF16, dict(strides=(68, 1)))),
    dict(x1=((6, 64), BF16, dict(strides=(56, 1)))), dict(x1=((6, 64), BF16, dict(strides=(-64, 1)))),
    dict(x1=((6, 64), BF16, dict(strides=(1, 6)))), dict(x1=((2, 3, 64), BF16, dict(strides=(640, 200, 1)))),
    dict(x1=((6, 64), BF16, dict(strides=(2 ** 32, 1)))), dict(x1=((6, 64), BF16, dict(data=FAKE + 8))),
    dict(x1=((2 ** 31 - 1, 2 ** 31 - 1, 64), BF16)), dict(x1=((6, 64), BF16, dict(fmt=W.FORMAT_PACKED))),
    dict(a=((3, 16, 96), BF16)), dict(a=((3, 12, 64), BF16), b=((3, 96, 12), BF16)),
    dict(a=((3, 136, 64), BF16), b=((3, 96, 136), BF16)), dict(a=((3, 0, 64), BF16), b=((3, 96, 0), BF16)),
    dict(a=((16, 64), BF16)), dict(a=((3, 16, 64), BF16, dict(strides=(2048, 64, 1)))),
    dict(a=((2049, 16, 64), BF16), b=((2049, 96, 16), BF16), scale=None, offsets=((2050,), I32)),
    dict(b=((2, 96, 16), BF16)), dict(b=((3, 96, 8), BF16)), dict(b=((3, 80, 16), BF16), y=None, out=((6, 80), BF16)),
    dict(b=((3, 96, 16), BF16, dict(data=FAKE + 2))), dict(scale=((2,), F32)), dict(scale=((3,), BF16)),
    dict(offsets=((3,), I32)), dict(offsets=((4,), W.DT_I64)), dict(source=((5,), I32)),
    dict(source=((6, 1), I32)), dict(y=((6, 64), BF16)), dict(y=((5, 96), BF16)), dict(y=((6, 96), F16)),
    dict(out=((6, 64), BF16)), dict(out=((6, 96), F32)), dict(y=((6, 96), BF16), out=((6, 96), BF16, dict(strides=(104, 1))))])
def test_add_refuses(kw):
    assert add(**kw)[0] == INVALID
    assert W.wqmm_last_error()


GRAD = dict(grad=((6, 96), BF16), x1=((6, 64), BF16), a=((3, 16, 64), BF16), b=((3, 96, 16), BF16), scale=((3,), F32),
            offsets=((4,), I32), source=((6,), I32), gx_in=((6, 64), BF16), gx=((6, 64), BF16),
            ga=((3, 16, 64), BF16), gb=((3, 96, 16), BF16))


def grad(**kw):
    t = {**GRAD, **kw}
    return call(W.lora_grad_get_workspace_size, *(t[n] for n in GRAD))


def test_grad_arguments():
    st, ws = grad()
    assert st == 0 and ws >= 2 * 6 * 2 * 16 * 2
    assert grad(gx_in=None)[0] == 0 and grad(gx_in=None, gx=None)[0] == 0 and grad(scale=None)[0] == 0
    assert grad(gx=None)[0] == NULL  # an addend without a result
    for name in ("grad", "x1", "a", "b", "offsets", "source", "ga", "gb"):
        assert grad(**{name: None})[0] == NULL, name
    for kw in (dict(grad=((6, 64), BF16)), dict(grad=((6, 96), F16)), dict(gx=((6, 96), BF16)),
               dict(gx_in=((5, 64), BF16)), dict(ga=((3, 64, 16), BF16)), dict(ga=((3, 16, 64), F32)),
               dict(gb=((3, 96, 16), BF16, dict(strides=(1600, 16, 1)))), dict(gb=((96, 16), BF16)),
               dict(gx=((6, 64), BF16, dict(strides=(72, 1)))),
               dict(ga=((2 ** 31 - 1, 2 ** 31 - 1, 2 ** 31 - 1), BF16))):
        assert grad(**kw)[0] == INVALID, kw


def test_null_pointers():
    for name in ("x1", "a", "b", "offsets", "source", "out"):
        assert add(**{name: None})[0] == NULL, name
        shape, dtype = ADD[name][:2]
        assert add(**{name: (shape, dtype, dict(data=0))}, **({} if name != "out" else dict(y=None)))[0] == NULL, name


def test_executors_are_one_shot_and_of_their_own_kind():
    t = {**ADD, "x1": ((5000, 64), BF16), "a": ((3, 32, 64), BF16), "b": ((3, 96, 32), BF16), "source": ((5000,), I32),
         "y": ((5000, 96), BF16), "out": ((5000, 96), BF16)}
    args = [T(*t[n]) for n in ("x1", "a", "b", "scale", "offsets", "source", "y", "out")]
    st, ws, ex = W.lora_get_workspace_size(*args)
    assert st == 0
    assert W.route_run(0, 0, ex, 0) == W.ERR_EXECUTOR
    assert W.lora_run(0, ws, ex, 0) == W.ERR_WORKSPACE  # a workspace is needed: refused, and consumed
    assert W.lora_run(FAKE, ws, ex, 0) == W.ERR_EXECUTOR


def test_wrappers_refuse():
    torch = pytest.importorskip("torch")
    x = torch.zeros(6, 64, dtype=torch.bfloat16)
    a, b = torch.zeros(3, 16, 64, dtype=torch.bfloat16), torch.zeros(3, 96, 16, dtype=torch.bfloat16)
    order = TokenOrder(torch.zeros(4, dtype=torch.int32), torch.zeros(6, dtype=torch.int32), None)
    for f in (lambda: lora.lora_add(x, a, b, order), lambda: lora.adapter_order(torch.zeros(6, dtype=torch.int32), 3),
              lambda: lora.lora_grad(torch.zeros(6, 96), x, a, b, order),
              lambda: lora.lora_weight_quant_matmul(x, W.desc(a[0]), None, a, b, order)):
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


def run_at(phase1, names, table, at, **kw):
    """Phase 2's status with tensor i at BIG * (i + 1), or where `at` says (bytes from there)."""
    t = {**table, **kw}
    descs = []
    for i, n in enumerate(names):
        if t[n] is None:
            descs.append(None)
            continue
        base, off = at.get(n, (n, 0))
        extra = t[n][2] if len(t[n]) > 2 else {}
        descs.append(T(*t[n][:2], data=BIG * (names.index(base) + 1) + off, **extra))
    st, ws, ex = phase1(*descs)
    assert st == 0, W.wqmm_last_error()
    return W.lora_run(BIG * 64, ws, ex, 0)


ADD_NAMES = ["x1", "a", "b", "scale", "offsets", "source", "y", "out"]
SQUARE = dict(x1=((6, 64), BF16), b=((3, 64, 16), BF16), y=((6, 64), BF16), out=((6, 64), BF16))
WIDE = lambda ld, n=64: ((6, n), BF16, dict(strides=(ld, 1)))


@no_gpu
@pytest.mark.parametrize("at,kw", [
    (dict(out=("x1", 0)), {}),  # k and n differ
    (dict(out=("x1", 0)), dict(SQUARE, x1=WIDE(128))), (dict(out=("x1", 0)), dict(SQUARE, out=WIDE(128))),
    (dict(out=("x1", 16)), SQUARE), (dict(out=("x1", 128)), SQUARE), (dict(out=("y", 16)), SQUARE),
    (dict(out=("y", 128)), SQUARE), (dict(y=("out", 128)), SQUARE), (dict(out=("x1", 6 * 128 - 16)), SQUARE),
    (dict(out=("x1", 112)), dict(SQUARE, x1=WIDE(128), out=WIDE(128))),  # columns of one matrix, eight in common
    (dict(x1=("out", 144)), dict(SQUARE, x1=WIDE(128), out=WIDE(128))),  # reaches into the next row's
    (dict(out=("a", 32)), {}), (dict(out=("b", 0)), {}), (dict(out=("scale", 0)), {}), (dict(out=("offsets", 0)), {}),
    (dict(source=("out", 1136)), {}), (dict(out=("x1", 0)), dict(x1=((1, 64), BF16), source=((1,), I32),
                                                              y=((1, 96), BF16), out=((1, 96), BF16)))])
def test_add_refuses_memory_in_common(at, kw):
    assert run_at(W.lora_get_workspace_size, ADD_NAMES, ADD, at, **kw) == INVALID
    assert "shares memory" in W.wqmm_last_error()


GRAD_SQUARE = dict(grad=((6, 64), BF16), b=((3, 64, 16), BF16), gb=((3, 64, 16), BF16))


@no_gpu
@pytest.mark.parametrize("at,kw", [
    (dict(gx=("grad", 0)), {}), (dict(gx=("x1", 16)), GRAD_SQUARE), (dict(gx=("grad", 16)), GRAD_SQUARE),
    (dict(gx=("x1", 0)), dict(GRAD_SQUARE, gx=WIDE(72), gx_in=None)),
    (dict(gx=("grad", 0)), dict(GRAD_SQUARE, grad=WIDE(72))), (dict(gx=("gx_in", 128)), {}),
    (dict(gx=("a", 0)), {}), (dict(ga=("a", 0)), {}), (dict(gb=("b", 0)), {}), (dict(ga=("x1", 0)), {}),
    (dict(gb=("grad", 64)), {}), (dict(ga=("gb", 16)), {}), (dict(gx=("ga", 16)), {}), (dict(gb=("gx_in", 0)), {}),
    (dict(ga=("source", 0)), {}), (dict(ga=("scale", 0)), {})])
def test_grad_refuses_memory_in_common(at, kw):
    assert run_at(W.lora_grad_get_workspace_size, list(GRAD), GRAD, at, **kw) == INVALID
    assert "shares memory" in W.wqmm_last_error()


def test_rows_of_the_gradients():
    """One CTA may go through all rows of an adapter while others wait, for a bounded time: fewer rows than forward."""
    rows = lambda m: {n: ((m, GRAD[n][0][1]), BF16) for n in ("grad", "x1", "gx_in", "gx")} | dict(source=((m,), I32))
    assert grad(**rows(2 ** 24))[0] == 0
    assert grad(**rows(2 ** 24 + 1))[0] == INVALID and "rows" in W.wqmm_last_error()
    assert grad(**rows(2 ** 26))[0] == INVALID
    assert add(x1=((2 ** 26, 64), BF16), source=((2 ** 26,), I32), y=None, out=((2 ** 26, 96), BF16))[0] == 0
    assert add(x1=((2 ** 26 + 1, 64), BF16), source=((2 ** 26 + 1,), I32), y=None, out=((2 ** 26 + 1, 96), BF16))[0] == INVALID


def test_flags_without_a_truth_value():
    """The error of a flag's own truth value is what the caller gets."""
    torch = pytest.importorskip("torch")
    x, a, b = torch.zeros(6, 64), torch.zeros(3, 16, 64), torch.zeros(3, 96, 16)
    i = torch.zeros(6, dtype=torch.int32)
    both = torch.tensor([True, False])
    for need, in_place in ((both, False), (True, both)):
        with pytest.raises(RuntimeError, match="Boolean value"):
            W.binding().lora_grad(torch.zeros(6, 96), x, a, b, None, i, i, x, need, in_place)
