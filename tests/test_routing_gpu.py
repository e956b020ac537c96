"""Token routing on the GPU against plain implementations: the sort against a host sort, sums in 64 bits."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import workloads as WL
import weight_quantized_gemm_anti_b200 as W
from weight_quantized_gemm_anti_b200 import routing as R

pytestmark = pytest.mark.gpu

TYPES = [torch.bfloat16, torch.float16, torch.float32]
U32 = 2.0 ** -24  # half a step of float32, relative


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    W.build()
    yield
    torch.cuda.synchronize()


def host_order(ids, groups):
    flat = ids.cpu().numpy().reshape(-1).astype(np.int64)
    key = np.where((flat >= 0) & (flat < groups), flat, groups)
    source = np.argsort(key, kind="stable")
    position = np.full(flat.size, -1)
    valid = int((key < groups).sum())
    position[source[:valid]] = np.arange(valid)
    offsets = np.concatenate([[0], np.cumsum(np.bincount(key, minlength=groups + 1)[:groups])])
    return offsets, source, position.reshape(tuple(ids.shape))


def check_order(order, ids, groups):
    for got, want in zip(order, host_order(ids, groups)):
        assert got.dtype == torch.int32
        assert np.array_equal(got.cpu().numpy(), want)


def make_ids(shape, groups, dtype=torch.int32, drop=0.1, seed=0):
    g = torch.Generator().manual_seed(seed)
    ids = torch.randint(0, groups, shape, generator=g)
    ids[torch.rand(shape, generator=g) < drop] = -1
    return ids.to(dtype).cuda()


def randn(*shape, dtype, seed=0, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).to(dtype).cuda()


# ------------------------------------------------------------------ sort
@pytest.mark.parametrize("slots", [0, 1, 31, 32, 33, 127, 1000, 4096, 4097, 9999, 70001, 300000])
@pytest.mark.parametrize("groups", [1, 2, 7, 256, 2048])
def test_sort(slots, groups):
    ids = make_ids((slots,), groups, torch.int32 if slots % 2 else torch.int64, seed=slots + groups)
    check_order(R.sort_tokens(ids, groups), ids, groups)


@pytest.mark.parametrize("shape", [(5, 3), (2, 7, 4), (0, 4), (4, 0), (1000, 8)])
def test_sort_shapes(shape):
    ids = make_ids(shape, 9)
    order = R.sort_tokens(ids, 9)
    assert tuple(order.position.shape) == shape
    check_order(order, ids, 9)


@pytest.mark.parametrize("slots", [100, 20000])
def test_sort_extremes(slots):
    all_one = torch.full((slots,), 3, dtype=torch.int64, device="cuda")
    check_order(R.sort_tokens(all_one, 5), all_one, 5)
    none = torch.full((slots,), -1, dtype=torch.int32, device="cuda")
    check_order(R.sort_tokens(none, 5), none, 5)
    # ids whose low 32 bits would name an expert, and the types' extremes
    wide = torch.tensor([2 ** 32 + 1, -2 ** 63, 2 ** 63 - 1, 4, 5, 0, -2 ** 32], device="cuda").repeat(slots // 7)
    check_order(R.sort_tokens(wide, 5), wide, 5)


# ------------------------------------------------------------------ dispatch
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32, torch.int8, torch.float8_e4m3fn, torch.int64])
@pytest.mark.parametrize("tokens,top,hidden", [(1, 1, 1), (3, 2, 7), (33, 4, 40), (257, 3, 1000), (5, 8, 8192),
                                               (1500, 2, 4096)])
def test_dispatch(dtype, tokens, top, hidden):
    ids = make_ids((tokens, top), 5, seed=hidden)
    order = R.sort_tokens(ids, 5)
    x = torch.randint(0, 100, (tokens, hidden)).float().to(dtype).cuda()
    out = torch.full((tokens * top + 2, hidden), 7, device="cuda").to(dtype)
    got = R.dispatch_tokens(x, order, out=out)
    assert got is out
    offsets, source, _ = host_order(ids, 5)
    want = np.full((tokens * top + 2, hidden), 7.0)
    n = offsets[-1]
    want[:n] = x.cpu().double().numpy()[source[:n] // top]
    assert np.array_equal(got.cpu().double().numpy(), want)  # the rows behind the last expert among them
    assert torch.equal(R.dispatch_tokens(x, order).view(torch.uint8)[:n], got.view(torch.uint8)[:n])


def test_dispatch_into_fewer_rows_and_off_alignment():
    ids = make_ids((50, 2), 4, drop=0)
    order = R.sort_tokens(ids, 4)
    for hidden, skip in ((24, 1), (24, 2), (24, 4), (17, 1)):
        x = randn(50 * hidden + 8, dtype=torch.float16)[skip:skip + 50 * hidden].view(50, hidden)
        buf = torch.zeros(64 * hidden + 8, dtype=torch.float16, device="cuda")
        out = buf[skip:skip + 60 * hidden].view(60, hidden)
        R.dispatch_tokens(x, order, out=out)
        _, source, _ = host_order(ids, 4)
        assert np.array_equal(out.cpu().numpy(), x.cpu().numpy()[source[:60] // 2])
        assert not buf[:skip].any() and not buf[skip + 60 * hidden:].any()


# ------------------------------------------------------------------ combine
def combine64(xs, position, weights, x3):
    """The sum in 64 bits and the sum of the terms' sizes."""
    xs, p = xs.cpu().double(), position.cpu().reshape(-1, position.shape[-1] if position.dim() > 1 else 1).long()
    w = torch.ones(p.shape, dtype=torch.float64) if weights is None else weights.cpu().double().reshape(p.shape)
    y = torch.zeros(p.shape[0], xs.shape[1], dtype=torch.float64)
    if x3 is not None:
        y += x3.cpu().double().reshape(y.shape)
    size = y.abs()
    for j in range(p.shape[1]):
        has = (p[:, j] >= 0) & (p[:, j] < xs.shape[0])
        term = w[has, j][:, None] * xs[p[has, j]]
        y[has] += term
        size[has] += term.abs()
    return y, size


def check_sum(got, want, size, terms):
    """Each of the sum's terms + 1 float32 roundings is off by at most half a step of what it rounds, at most U32 of
    the terms' sizes; then one rounding to the type (half a step of the type, at least half its smallest number)."""
    acc = (terms + 1) * U32 * size * 1.01
    half = torch.finfo(got.dtype).eps / 2
    tiny = torch.finfo(got.dtype).smallest_normal * torch.finfo(got.dtype).eps / 2
    err = (got.cpu().double().reshape(want.shape) - want).abs()
    assert bool((err <= acc + half * (want.abs() + acc) + tiny).all()), float(err.max())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("tokens,top,hidden", [(1, 1, 8), (3, 2, 7), (33, 5, 40), (130, 9, 1001), (16, 2, 4096),
                                               (700, 4, 2048)])
@pytest.mark.parametrize("with_x3", [False, True])
def test_combine(dtype, tokens, top, hidden, with_x3):
    ids = make_ids((tokens, top), 6, drop=0.3, seed=tokens)
    order = R.sort_tokens(ids, 6)
    xs = randn(tokens * top, hidden, dtype=dtype, seed=1)
    x3 = randn(tokens, hidden, dtype=dtype, seed=2) if with_x3 else None
    for wt in (torch.float32, torch.bfloat16, torch.float16, None):
        w = None if wt is None else (torch.rand(tokens, top, generator=torch.Generator().manual_seed(3)) + 0.1).to(wt).cuda()
        got = R.combine_tokens(xs, order, w, x3=x3)
        assert got.dtype == dtype and tuple(got.shape) == (tokens, hidden)
        check_sum(got, *combine64(xs, order.position, w, x3), terms=top + 1)


def test_combine_skips_what_is_dropped():
    """Rows of no slot, their weights and positions out of range are not read: no NaN of theirs reaches a sum."""
    position = torch.tensor([[0, -1], [-1, -1], [2, 99], [1, -2 ** 31], [3, 2 ** 31 - 1]], dtype=torch.int32).cuda()
    xs = randn(6, 64, dtype=torch.bfloat16)
    xs[4:] = float("nan")
    w = torch.ones(5, 2, device="cuda")
    w[position.reshape(5, 2) < 0] = float("nan")
    w[2, 1] = w[4, 1] = float("inf")
    order = R.TokenOrder(None, None, position)
    got = R.combine_tokens(xs, order, w)
    want = torch.stack([xs[0], torch.zeros_like(xs[0]), xs[2], xs[1], xs[3]])
    assert torch.equal(got, want)
    xs[1, 3], xs[2, 5] = float("inf"), float("nan")  # values that are there do come through
    got = R.combine_tokens(xs, order, w)
    assert got[3, 3] == float("inf") and torch.isnan(got[2, 5]) and int(torch.isnan(got).sum()) == 1
    # the same row for two tokens, no rows at all, one choice per token, three dimensions
    both = R.TokenOrder(None, None, torch.tensor([[0, 0], [0, -1]], dtype=torch.int32).cuda())
    got = R.combine_tokens(xs, both)
    check_sum(got, *combine64(xs, both.position, None, None), terms=2)
    assert not R.combine_tokens(xs[:0], both).any()
    one = R.TokenOrder(None, None, torch.tensor([2, 0, 1], dtype=torch.int32).cuda())
    assert torch.equal(R.combine_tokens(xs[:, :1].contiguous(), one)[:, 0].float()[[0, 1]], xs[[2, 0], 0].float())
    x3 = torch.zeros(2, 2, 64, dtype=torch.bfloat16, device="cuda")
    got = R.combine_tokens(xs, R.TokenOrder(None, None, position[:4].reshape(2, 2, 2).contiguous()), x3=x3)
    assert got.shape == (2, 2, 64) and torch.equal(got[0, 0], xs[0])


# ------------------------------------------------------------------ gradients
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("tokens,top,hidden", [(1, 1, 8), (3, 2, 7), (33, 5, 40), (130, 9, 1001), (16, 2, 4096),
                                               (700, 4, 2048), (65, 17, 200)])
def test_combine_grad(dtype, tokens, top, hidden):
    ids = make_ids((tokens, top), 6, drop=0.3, seed=tokens)
    order = R.sort_tokens(ids, 6)
    xs = randn(tokens * top, hidden, dtype=dtype, seed=1)
    grad = randn(tokens, hidden, dtype=dtype, seed=2)
    wt = torch.float32 if hidden % 2 else dtype
    w = (torch.rand(tokens, top, generator=torch.Generator().manual_seed(3)) + 0.1).to(wt).cuda()
    out = torch.full_like(xs, 7)
    got_rows, got_w = R.combine_tokens_grad(grad, xs, order, w, out=out)
    assert got_rows is out and got_w.dtype == wt
    offsets, source, _ = host_order(ids, 6)
    n = int(offsets[-1])
    slot = torch.from_numpy(source[:n])
    g = grad.cpu().double()[slot // top]
    want = g * w.cpu().double().reshape(-1)[slot][:, None]
    check_sum(got_rows[:n], want, want.abs(), terms=0)  # one product, one rounding
    assert bool((got_rows[n:] == 7).all())
    terms = g * xs.cpu().double()[:n]
    dots = torch.zeros(tokens * top, dtype=torch.float64)
    sizes = torch.zeros_like(dots)
    dots[slot], sizes[slot] = terms.sum(1), terms.abs().sum(1)
    # a thread sums at most hidden / 32 + 8 products, then come five shuffles and at most eight warps
    check_sum(got_w.reshape(-1), dots, sizes, terms=hidden // 32 + 8 + 13)
    assert not got_w.reshape(-1).cpu()[torch.from_numpy(source[n:])].any()


def test_gradients_agree_with_differences():
    """Along random directions, in float32: f is linear in xs and in w, so a difference of any length is exact but
    for the roundings of f's two values, each term of them off by at most (terms + 1) U32 of its size."""
    tokens, top, hidden = 19, 3, 96
    order = R.sort_tokens(make_ids((tokens, top), 4, drop=0.2), 4)
    xs = randn(tokens * top, hidden, dtype=torch.float32, seed=1)
    w = randn(tokens, top, dtype=torch.float32, seed=2)
    c = randn(tokens, hidden, dtype=torch.float32, seed=3)
    rows, weights = R.combine_tokens_grad(c, xs, order, w, out=torch.zeros_like(xs))
    f = lambda xs, w: (R.combine_tokens(xs, order, w).double() * c.double()).sum()
    sizes = lambda xs, w: float((R.combine_tokens(xs.abs(), order, w.abs()).double() * c.double().abs()).sum())
    dx, dw = randn(tokens * top, hidden, dtype=torch.float32, seed=4), randn(tokens, top, dtype=torch.float32, seed=5)
    for at, step, by in (((xs + dx, w), dx, rows), ((xs, w + dw), dw, weights)):
        bound = 2 * (top + 2) * U32 * (sizes(*at) + sizes(xs, w)) * 1.01
        # the gradient's own roundings, and those of xs + dx
        bound += (hidden // 32 + 24) * U32 * (sizes(*at) + sizes(xs, w)) * 2
        assert abs(float(f(*at) - f(xs, w)) - float((by.double() * step.double()).sum())) <= bound


def test_dispatch_gradient_is_combine_without_weights():
    ids = make_ids((40, 3), 5, drop=0.3)
    order = R.sort_tokens(ids, 5)
    grad = randn(120, 72, dtype=torch.bfloat16)
    got = R.combine_tokens(grad, order)
    check_sum(got, *combine64(grad, order.position, None, None), terms=3)


# ------------------------------------------------------------------ streams, graphs, the operators together
def test_streams_and_graphs():
    ids = make_ids((3000, 4), 16)
    x = randn(3000, 256, dtype=torch.bfloat16)
    w = torch.rand(3000, 4, device="cuda")

    def step(stream=None):
        order = R.sort_tokens(ids, 16, stream=stream)
        rows = R.dispatch_tokens(x, order, stream=stream)
        return order, R.combine_tokens(rows, order, w, x3=x, stream=stream)

    order, want = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    _, got = step(side)
    _, raw = step(side.cuda_stream)
    side.synchronize()
    assert torch.equal(got, want) and torch.equal(raw, want)
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            held = step()
        graphs.append((g, held))
    ids.copy_(make_ids((3000, 4), 16, seed=9))
    new_order, new = step()
    for g, held in graphs + graphs:
        g.replay()
        assert torch.equal(held[1], new)
        for a, b in zip(held[0], new_order):
            assert torch.equal(a, b)
    assert not torch.equal(new, want)


def test_runs_are_bitwise_equal():
    ids = make_ids((2000, 6), 32, drop=0.1)
    xs, grad = randn(12000, 1024, dtype=torch.bfloat16), randn(2000, 1024, dtype=torch.bfloat16, seed=1)
    w = torch.rand(2000, 6, device="cuda")
    order = R.sort_tokens(ids, 32)
    first = None
    for _ in range(5):
        out = torch.zeros_like(xs)
        got = (*R.sort_tokens(ids, 32), R.combine_tokens(xs, order, w),
               *R.combine_tokens_grad(grad, xs, order, w, out=out))
        first = first or got
        assert all(torch.equal(a, b) for a, b in zip(first, got))


def test_experts_of_quantised_weights():
    """sort, dispatch, the experts' anti-quant products and combine, as a mixture of experts uses them."""
    tokens, top, hidden, n, experts = 37, 2, 128, 64, 5
    ids = make_ids((tokens, top), experts, drop=0.1)
    ids[ids == 3] = 1  # an expert without rows
    order = R.sort_tokens(ids, experts)
    x = randn(tokens, hidden, dtype=torch.bfloat16)
    w = torch.rand(tokens, top, device="cuda")
    qs = [torch.randint(-128, 128, (hidden, n), dtype=torch.int8, generator=torch.Generator().manual_seed(e)).cuda()
          for e in range(experts)]
    scales = [torch.full((n,), 0.002 * (e + 1), dtype=torch.bfloat16, device="cuda") for e in range(experts)]
    rows = R.dispatch_tokens(x, order)
    y = R.expert_weight_quant_matmul(rows, order, [W.desc(q) for q in qs], scales)
    got = R.combine_tokens(y, order, w)
    want = torch.zeros(tokens, n, dtype=torch.float64)
    size = torch.zeros_like(want)
    for e in range(experts):
        weight = qs[e].cpu().double() * scales[e].cpu().double()
        for t, j in (ids.cpu() == e).nonzero().tolist():
            out = x[t].cpu().double() @ weight
            want[t] += float(w[t, j]) * out
            size[t] += float(w[t, j]) * (x[t].cpu().double().abs() @ weight.abs())
    # of each term: the weight rounded to bf16 once, the product's row rounded to bf16 once, 32-bit sums of
    # `hidden` products; then the result's rounding
    half = 2.0 ** -8
    bound = size * (2 * half + (hidden + 4) * U32) * 1.02 + half * want.abs()
    assert bool(((got.cpu().double() - want).abs() <= bound).all())


@pytest.mark.parametrize("tokens,top,hidden", [(33, 5, 40), (130, 9, 1001), (700, 4, 2048)])
def test_results_in_place(tokens, top, hidden):
    """The addend as combine's result, the experts' rows as their own gradient; other sharing is refused."""
    ids = make_ids((tokens, top), 6, drop=0.3, seed=tokens)
    order = R.sort_tokens(ids, 6)
    xs, x3 = randn(tokens * top, hidden, dtype=torch.bfloat16, seed=1), randn(tokens, hidden, dtype=torch.bfloat16, seed=2)
    w = torch.rand(tokens, top, device="cuda")
    want = R.combine_tokens(xs, order, w, x3=x3)
    y = x3.clone()
    assert R.combine_tokens(xs, order, w, x3=y, out=y) is y and torch.equal(y, want)
    rows, weights = R.combine_tokens_grad(x3, xs, order, w, out=xs.clone())
    z = xs.clone()
    got = R.combine_tokens_grad(x3, z, order, w, out=z)
    assert got[0] is z and torch.equal(z, rows) and torch.equal(got[1], weights)
    for f in (lambda: R.combine_tokens(xs, order, w, out=xs[:tokens]),
              lambda: R.combine_tokens_grad(xs[:tokens], z, order, w, out=xs),
              lambda: R.dispatch_tokens(xs[:tokens], order, out=xs)):
        with pytest.raises(W.WqmmError, match="shares memory"):
            f()


def expert_case(tokens=37, top=2, hidden=128, n=64, experts=5):
    ids = make_ids((tokens, top), experts, drop=0.1)
    order = R.sort_tokens(ids, experts)
    rows = R.dispatch_tokens(randn(tokens, hidden, dtype=torch.bfloat16), order)
    qs = [torch.randint(-128, 128, (hidden, n), dtype=torch.int8, generator=torch.Generator().manual_seed(e)).cuda()
          for e in range(experts)]
    scales = [torch.full((n,), 0.002 * (e + 1), dtype=torch.bfloat16, device="cuda") for e in range(experts)]
    return order, rows, qs, [W.desc(q) for q in qs], scales


def test_experts_refuse():
    order, rows, qs, descs, scales = expert_case()
    out = torch.full((rows.shape[0], 64), 3.0, device="cuda").bfloat16()
    bounds = order.offsets.tolist()
    down = [bounds[0], bounds[2], bounds[1], *bounds[3:]]
    for kw in (dict(x2_descs=[]), dict(x2_descs=descs[:4]), dict(antiquant_scales=scales[:4]),
               dict(antiquant_scales=scales + scales[:1]), dict(antiquant_offsets=scales[:2]), dict(biases=scales[:3]),
               dict(bounds=bounds[:-1]), dict(bounds=[0]), dict(bounds=down), dict(bounds=[-1, *bounds[1:]]),
               dict(out=out[:bounds[-1] - 1]), dict(out=out[0]), dict(x_sorted=rows.view(2, -1, 128))):
        with pytest.raises(ValueError):
            R.expert_weight_quant_matmul(**{**dict(x_sorted=rows, order=order, x2_descs=descs,
                                                   antiquant_scales=scales, out=out, bounds=bounds), **kw})
        assert bool((out == 3).all()), kw
    square = [torch.randint(-128, 128, (128, 128), dtype=torch.int8, device="cuda") for _ in qs]
    wide = [torch.full((128,), 0.002, dtype=torch.bfloat16, device="cuda") for _ in qs]
    before = rows.clone()
    with pytest.raises(ValueError, match="shares memory"):
        R.expert_weight_quant_matmul(rows, order, [W.desc(q) for q in square], wide, out=rows)
    assert torch.equal(rows.view(torch.int16), before.view(torch.int16))  # as bits: rows of no slot hold anything


@pytest.mark.parametrize("kept", [0, 1, 20, 50, 74])
def test_experts_of_fewer_rows_than_slots(kept):
    """Rows up to a capacity: what lies behind is dropped, whole experts among it."""
    order, rows, _, descs, scales = expert_case()
    want = R.expert_weight_quant_matmul(rows, order, descs, scales)
    end = min(kept, int(order.offsets[-1]))
    for bounds in (None, order.offsets.tolist()):
        got = R.expert_weight_quant_matmul(rows[:kept], order, descs, scales, bounds=bounds)
        assert tuple(got.shape) == (kept, 64) and torch.equal(got[:end], want[:end])
