"""Low-rank adapters on the GPU against their formulas in 64 bits."""
import pytest

torch = pytest.importorskip("torch")

import weight_quantized_gemm_anti_b200 as W
from weight_quantized_gemm_anti_b200 import lora
from weight_quantized_gemm_anti_b200.routing import TokenOrder

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    W.build()
    yield
    torch.cuda.synchronize()


class Case:
    """Random inputs of one problem; the rows' adapters in random order, some rows with none."""

    def __init__(self, m, k, n, rank, adapters, dtype, bare=0.2, seed=0, x_std=1.0, a_std=None, b_std=0.1, grad_std=1.0):
        g = torch.Generator().manual_seed(seed)
        dt = TYPES[dtype]
        r = lambda *s, std=1.0: (torch.randn(s, generator=g) * std).to(dt).cuda()
        self.ids = torch.randint(0, adapters, (m,), generator=g)
        self.ids[torch.rand(m, generator=g) < bare] = -1
        self.x, self.y, self.grad = r(m, k, std=x_std), r(m, n), r(m, n, std=grad_std)
        self.gx = r(m, k, std=grad_std)
        self.a, self.b = r(adapters, rank, k, std=a_std or k ** -0.5), r(adapters, n, rank, std=b_std)
        self.scale = (torch.rand(adapters, generator=g) + 0.5).cuda()
        self.order = lora.adapter_order(self.ids.cuda(), adapters)


def exact(x, a, b, ids, scale, y):
    """The sum, and the size of what it sums: the absolute values of all products."""
    x, a, b = x.cpu().double(), a.cpu().double(), b.cpu().double()
    out = torch.zeros(x.shape[0], b.shape[1], dtype=torch.float64) if y is None else y.cpu().double().clone()
    size = torch.zeros_like(out)
    for i in range(a.shape[0]):
        at = (ids == i).nonzero()[:, 0]
        s = 1.0 if scale is None else float(scale[i])
        out[at] += s * (x[at] @ a[i].T) @ b[i].T
        size[at] += s * (x[at].abs() @ a[i].abs().T) @ b[i].abs().T
    return out, size


def exact_grad(grad, x, a, b, ids, scale, gx):
    grad, x, a, b = (t.cpu().double() for t in (grad, x, a, b))
    out = torch.zeros_like(x) if gx is None else gx.cpu().double().clone()
    da, db, sx, sa, sb = (torch.zeros_like(t) for t in (a, b, x, a, b))
    for i in range(a.shape[0]):
        at = (ids == i).nonzero()[:, 0]
        s = 1.0 if scale is None else float(scale[i])
        out[at] += s * (grad[at] @ b[i]) @ a[i]
        sx[at] += s * (grad[at].abs() @ b[i].abs()) @ a[i].abs()
        da[i], sa[i] = s * (grad[at] @ b[i]).T @ x[at], s * (grad[at].abs() @ b[i].abs()).T @ x[at].abs()
        db[i], sb[i] = s * grad[at].T @ (x[at] @ a[i].T), s * grad[at].abs().T @ (x[at].abs() @ a[i].abs().T)
    return (out, sx), (da, sa), (db, sb)


def check(got, want, size, first, second, addend=None):
    """``first`` and ``second``: the lengths of the two contractions.  A matrix instruction adds 16 products to its
    sum and keeps at least 22 bits of the largest, so a contraction of length L is off by at most (L / 16 + 8) *
    2^-22 of its products' sizes (the 8: the shares' sums).  The value between the two is kept as two 16-bit
    numbers, off by at most the square of half a step (bfloat16 2^-16; float16 2^-22, and less than 2^-38 of its
    row's largest).  The second contraction runs over both numbers.  At the end one rounding to the type."""
    half = torch.finfo(got.dtype).eps / 2
    rel = (first / 16 + 8 + 2 * second / 16 + 8) * 2.0 ** -22 + half * half * 1.01 + 4 * 2.0 ** -24
    slack = size * rel
    if addend is not None:
        slack = slack + addend.cpu().double().abs() * 2.0 ** -23
    tiny = torch.finfo(got.dtype).smallest_normal * torch.finfo(got.dtype).eps / 2
    err = (got.cpu().double().reshape(want.shape) - want).abs()
    bad = err > slack + half * (want.abs() + slack) + tiny
    assert not bool(bad.any()), (float(err.max()), int(bad.sum()), bad.nonzero()[:4].tolist())


SHAPES = [(1, 32, 32, 1), (5, 96, 160, 3), (16, 512, 256, 16), (17, 1056, 96, 2), (64, 128, 416, 1), (65, 64, 128, 40),
          (130, 256, 128, 2), (300, 640, 288, 5), (1000, 2048, 1024, 7)]
MANY = [(1100, 512, 96, 2), (2100, 1024, 416, 3), (4200, 96, 160, 5)]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("rank", [8, 16, 24, 64, 72, 128])
@pytest.mark.parametrize("shape", SHAPES + MANY, ids=str)
def test_add(dtype, rank, shape):
    m, k, n, adapters = shape
    c = Case(m, k, n, rank, adapters, dtype, seed=m + rank)
    got = lora.lora_add(c.x, c.a, c.b, c.order, c.scale, y=c.y)
    want, size = exact(c.x, c.a, c.b, c.ids, c.scale, c.y)
    check(got, want, size, k, rank, c.y)
    bare = c.ids < 0
    assert torch.equal(got.cpu()[bare], c.y.cpu()[bare])
    # without an addend, without a scale
    got = lora.lora_add(c.x, c.a, c.b, c.order)
    check(got, *exact(c.x, c.a, c.b, c.ids, None, None), k, rank)
    assert not got.cpu()[bare].any()
    # in place
    y = c.y.clone()
    assert lora.lora_add(c.x, c.a, c.b, c.order, c.scale, y=y, out=y) is y
    assert torch.equal(y, lora.lora_add(c.x, c.a, c.b, c.order, c.scale, y=c.y))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("rank", [8, 16, 24, 64, 72, 128])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_grad(dtype, rank, shape):
    m, k, n, adapters = shape
    c = Case(m, k, n, rank, adapters, dtype, seed=m + rank)
    got = lora.lora_grad(c.grad, c.x, c.a, c.b, c.order, c.scale, grad_x=c.gx)
    (dx, sx), (da, sa), (db, sb) = exact_grad(c.grad, c.x, c.a, c.b, c.ids, c.scale, c.gx)
    check(got[0], dx, sx, n, rank, c.gx)
    check(got[1], da, sa, n, m)
    check(got[2], db, sb, k, m)
    none = [i for i in range(adapters) if not (c.ids == i).any()]
    assert not got[1][none].any() and not got[2][none].any()
    again = lora.lora_grad(c.grad, c.x, c.a, c.b, c.order, need_grad_x=False)
    assert again[0] is None
    _, (da, sa), (db, sb) = exact_grad(c.grad, c.x, c.a, c.b, c.ids, None, None)
    check(again[1], da, sa, n, m)
    check(again[2], db, sb, k, m)
    gx = c.gx.clone()
    placed = lora.lora_grad(c.grad, c.x, c.a, c.b, c.order, c.scale, grad_x=gx, in_place=True)
    assert placed[0] is gx and torch.equal(gx, got[0])
    bare = lora.lora_grad(c.grad, c.x, c.a, c.b, c.order, c.scale)[0]
    check(bare, *exact_grad(c.grad, c.x, c.a, c.b, c.ids, c.scale, None)[0], n, rank)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_no_row_and_every_row_without_adapter(dtype):
    for ids in (torch.full((70,), -1), torch.full((70,), 1), torch.arange(70) % 64):
        c = Case(70, 64, 96, 16, 64, dtype)
        c.ids, c.order = ids, lora.adapter_order(ids.cuda(), 64)
        got = lora.lora_add(c.x, c.a, c.b, c.order, c.scale, y=c.y)
        check(got, *exact(c.x, c.a, c.b, ids, c.scale, c.y), 64, 16, c.y)
        for g, (want, size), lens in zip(lora.lora_grad(c.grad, c.x, c.a, c.b, c.order, c.scale, grad_x=c.gx),
                                         exact_grad(c.grad, c.x, c.a, c.b, ids, c.scale, c.gx),
                                         ((96, 16), (96, 70), (64, 70))):
            check(g, want, size, *lens, c.gx if g.shape == c.gx.shape else None)


@pytest.mark.parametrize("rows", [3, 100, 4200])
def test_strided_rows_and_three_dimensions(rows):
    """Slices of a fused projection: x1, y and the output are columns of wider matrices, whose others stay."""
    rank = 24 if rows > 4096 else 16
    c = Case(rows, 96, 128, rank, 3, "bf16")
    wide_x = torch.randn(rows, 96 + 40, device="cuda").bfloat16()
    wide_y, wide_o = torch.randn(rows, 400, device="cuda").bfloat16(), torch.full((rows, 264), 3.0, device="cuda").bfloat16()
    x, y, out = wide_x[:, 24:120], wide_y[:, 128:256], wide_o[:, 64:192]
    lora.lora_add(x, c.a, c.b, c.order, c.scale, y=y, out=out)
    check(out, *exact(x, c.a, c.b, c.ids, c.scale, y), 96, rank, y)
    assert bool((wide_o[:, :64] == 3).all()) and bool((wide_o[:, 192:] == 3).all())
    before = wide_y.clone()
    lora.lora_add(x, c.a, c.b, c.order, c.scale, y=y, out=y)
    assert torch.equal(y, out)
    assert torch.equal(wide_y[:, :128], before[:, :128]) and torch.equal(wide_y[:, 256:], before[:, 256:])
    gx, da, db = lora.lora_grad(out, x, c.a, c.b, c.order, c.scale)
    same = lora.lora_grad(out.contiguous(), x.contiguous(), c.a, c.b, c.order, c.scale)
    assert all(torch.equal(p, q) for p, q in zip((gx, da, db), same))
    if rows == 100:
        shape = lambda t: t.view(4, 25, -1)
        got = lora.lora_add(shape(c.x), c.a, c.b, c.order, c.scale, y=shape(c.y))
        assert got.shape == (4, 25, 128)
        assert torch.equal(got.view(100, 128), lora.lora_add(c.x, c.a, c.b, c.order, c.scale, y=c.y))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("m,rank", [(5, 16), (300, 16), (40, 128), (300, 64), (2100, 64), (4200, 24)])
def test_in_place_of_an_input(dtype, m, rank):
    """A residual: the input itself is the addend and the result, and the gradient of the result the input's."""
    c = Case(m, 288, 288, rank, 4, dtype, b_std=0.02)
    want = lora.lora_add(c.x, c.a, c.b, c.order, c.scale, y=c.x)
    x = c.x.clone()
    assert lora.lora_add(x, c.a, c.b, c.order, c.scale, y=x, out=x) is x
    assert torch.equal(x, want)
    want = lora.lora_grad(c.grad, c.x, c.a, c.b, c.order, c.scale, grad_x=c.grad)
    grad = c.grad.clone()
    got = lora.lora_grad(grad, c.x, c.a, c.b, c.order, c.scale, grad_x=grad, in_place=True)
    assert got[0] is grad and all(torch.equal(p, q) for p, q in zip(got, want))
    want = lora.lora_grad(c.grad, c.x, c.a, c.b, c.order, c.scale, grad_x=c.x)
    x = c.x.clone()
    got = lora.lora_grad(c.grad, x, c.a, c.b, c.order, c.scale, grad_x=x, in_place=True)
    assert all(torch.equal(p, q) for p, q in zip(got, want))


def test_values_that_are_not_finite_stay_in_their_rows():
    for dtype in ("bf16", "f16"):
        for m in (40, 200, 4200):
            c = Case(m, 128, 96, 24 if m > 4096 else 16, 3, dtype, bare=0.3)
            clean = lora.lora_add(c.x, c.a, c.b, c.order, c.scale, y=c.y)
            clean_grad = lora.lora_grad(c.grad, c.x, c.a, c.b, c.order, c.scale)
            bare = (c.ids < 0).nonzero()[:, 0].cuda()
            x, grad = c.x.clone(), c.grad.clone()
            x[bare], grad[bare] = float("nan"), float("inf")
            assert torch.equal(lora.lora_add(x, c.a, c.b, c.order, c.scale, y=c.y), clean)
            got = lora.lora_grad(grad, x, c.a, c.b, c.order, c.scale)
            assert all(torch.equal(p, q) for p, q in zip(got, clean_grad))
            hit = int((c.ids == 1).nonzero()[0, 0])
            x = c.x.clone()
            x[hit, 5] = float("inf")
            got = lora.lora_add(x, c.a, c.b, c.order, c.scale, y=c.y)
            assert not bool(torch.isfinite(got[hit]).any())
            rest = torch.arange(m) != hit
            assert torch.equal(got[rest.cuda()], clean[rest.cuda()])
            _, da, db = lora.lora_grad(c.grad, x, c.a, c.b, c.order, c.scale)
            others = [0, 2]
            assert torch.equal(da[others], clean_grad[1][others]) and torch.equal(db[others], clean_grad[2][others])
            assert not bool(torch.isfinite(da[1][:, 5]).any())


def test_float16_range():
    """x A^T beyond float16's largest number, and gradients below its smallest normal one: what is kept between the
    contractions reaches as far as 32 bits do."""
    for m in (12, 150, 4200):
        rank = 24 if m > 4096 else 16
        c = Case(m, 256, 96, rank, 2, "f16", x_std=2000.0, a_std=50.0, b_std=1e-6, grad_std=3e-5)
        assert float((c.x.float() @ c.a[0].float().T).abs().max()) > 7e5
        got = lora.lora_add(c.x, c.a, c.b, c.order, c.scale, y=c.y)
        check(got, *exact(c.x, c.a, c.b, c.ids, c.scale, c.y), 256, rank, c.y)
        got = lora.lora_grad(c.grad, c.x, c.a, c.b, c.order, c.scale, grad_x=c.gx)
        for g, (want, size), lens in zip(got, exact_grad(c.grad, c.x, c.a, c.b, c.ids, c.scale, c.gx),
                                         ((96, rank), (96, m), (256, m))):
            check(g, want, size, *lens, c.gx if g.shape == c.gx.shape else None)
        # rows of very different sizes in one adapter
        c.x[::2] *= 1e-3
        c.grad[1::3] *= 8e-3
        got = lora.lora_grad(c.grad, c.x, c.a, c.b, c.order, c.scale)
        for g, (want, size), lens in zip(got, exact_grad(c.grad, c.x, c.a, c.b, c.ids, c.scale, None),
                                         ((96, rank), (96, m), (256, m))):
            check(g, want, size, *lens)


def test_orders_that_name_no_row():
    """Entries of the order out of range are skipped: nothing is read or written for them."""
    for m in (6, 90, 4200):
        c = Case(m, 64, 96, 24 if m > 4096 else 16, 3, "bf16", bare=0)
        source = c.order.source.clone()
        gone = int(source[2])
        source[2] = m + 5
        order = TokenOrder(c.order.offsets, source, None)
        out = torch.full_like(c.y, 7)
        lora.lora_add(c.x, c.a, c.b, order, c.scale, y=c.y, out=out)
        want = lora.lora_add(c.x, c.a, c.b, c.order, c.scale, y=c.y)
        want[gone] = 7
        assert torch.equal(out, want)
        wild = TokenOrder(torch.tensor([-5, 2, 2 ** 31 - 1, -1], dtype=torch.int32, device="cuda"), source, None)
        lora.lora_add(c.x, c.a, c.b, wild, c.scale, y=c.y, out=out)
        lora.lora_grad(c.grad, c.x, c.a, c.b, wild, c.scale)
    torch.cuda.synchronize()


def test_gradients_agree_with_differences():
    """Along a random direction the result is linear in each of x, A and B: a central difference of a whole step is
    exact but for the result's bounds, which stand in ``check``; the products with c and their sum are in 64 bits."""
    c = Case(60, 128, 96, 16, 2, "f16", b_std=0.05)
    dx, da, db = lora.lora_grad(c.grad, c.x, c.a, c.b, c.order, c.scale)
    f = lambda x, a, b: (exact(x, a, b, c.ids, c.scale, None)[0] * c.grad.cpu().double()).sum()
    for name, by in (("x", dx), ("a", da), ("b", db)):
        at = {"x": c.x.cpu().double(), "a": c.a.cpu().double(), "b": c.b.cpu().double()}
        step = torch.randn(at[name].shape, generator=torch.Generator().manual_seed(3)).double()
        plus, minus = ({**at, name: at[name] + s * step} for s in (1, -1))
        diff = float(f(**plus) - f(**minus)) / 2
        # each element of the gradient is off by half a step of its own, and the bound of its sums
        want = dict(zip("xab", exact_grad(c.grad, c.x, c.a, c.b, c.ids, c.scale, None)))[name]
        slack = float(((2.0 ** -11 * want[0].abs() + 2.0 ** -15 * want[1]) * step.abs()).sum())
        assert abs(diff - float((by.cpu().double() * step).sum())) <= slack


def test_streams_graphs_and_repeats():
    for m, adapters in ((12, 8), (500, 3), (4200, 3)):
        c = Case(m, 512, 256, 24 if m > 4096 else 16, adapters, "bf16")
        step = lambda s=None: (lora.lora_add(c.x, c.a, c.b, c.order, c.scale, y=c.y, stream=s),
                               *lora.lora_grad(c.grad, c.x, c.a, c.b, c.order, c.scale, grad_x=c.gx, stream=s))
        want = step()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        for s in (side, side.cuda_stream):
            got = step(s)
            side.synchronize()
            assert all(torch.equal(p, q) for p, q in zip(got, want))
        graphs = []
        for _ in range(2):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                held = step()
            graphs.append((g, held))
        c.x.mul_(0.5)
        want = step()
        for _ in range(3):
            for g, held in graphs:
                g.replay()
                assert all(torch.equal(p, q) for p, q in zip(held, want))


@pytest.mark.parametrize("ranks", [(16, 64), (64, 128), (24, 24), (128, 8)], ids=str)
def test_two_streams_at_once(ranks):
    """Calls of two streams side by side, few and many rows in turn: no call sees another's workspace or sums."""
    work = []
    for i, rank in enumerate(ranks):
        cases = [Case(m, 512, 640, rank, 3, ("bf16", "f16")[i], seed=i) for m in (20, 1500, 4200)]
        step = lambda c: (lora.lora_add(c.x, c.a, c.b, c.order, c.scale, y=c.y),
                          *lora.lora_grad(c.grad, c.x, c.a, c.b, c.order, c.scale, grad_x=c.gx))
        work.append((torch.cuda.Stream(), cases, step, [step(c) for c in cases]))
    torch.cuda.synchronize()
    got = [[] for _ in work]
    for turn in range(8):
        for (stream, cases, step, _), out in zip(work, got):
            with torch.cuda.stream(stream):
                out.append([step(c) for c in cases])
    torch.cuda.synchronize()
    for (_, _, _, want), out in zip(work, got):
        for turn in out:
            for p, q in zip(turn, want):
                assert all(torch.equal(u, v) for u, v in zip(p, q))


def test_beside_a_quantised_projection():
    m, k, n = 37, 256, 128
    c = Case(m, k, n, 16, 4, "bf16")
    q = torch.randint(-128, 128, (k, n), dtype=torch.int8, generator=torch.Generator().manual_seed(1)).cuda()
    s = torch.full((n,), 0.002, dtype=torch.bfloat16, device="cuda")
    got = lora.lora_weight_quant_matmul(c.x, W.desc(q), s, c.a, c.b, c.order, c.scale, x3=c.y)
    base = W.weight_quant_matmul(c.x, W.desc(q), s, x3=c.y)
    check(got, *exact(c.x, c.a, c.b, c.ids, c.scale, base), k, 16, base)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    same = lora.lora_weight_quant_matmul(c.x, W.desc(q), s, c.a, c.b, c.order, c.scale, x3=c.y, stream=side)
    side.synchronize()
    assert torch.equal(got, same)


@pytest.mark.parametrize("m", [40, 600, 4200])
def test_chains_of_calls_see_each_others_results(m):
    """Calls that follow each other with nothing between, each reading what the one before wrote: in place on one
    tensor, with an order sorted anew into the same memory, and as a replayed graph."""
    c = Case(m, 256, 640, 24 if m > 4096 else 16, 5, "bf16", b_std=0.02)
    ids = [torch.randint(-1, 5, (m,), generator=torch.Generator().manual_seed(s)).cuda() for s in range(4)]
    want = c.y.clone()
    for i in range(24):
        order = lora.adapter_order(ids[i % 4], 5)
        torch.cuda.synchronize()
        want = lora.lora_add(c.x, c.a, c.b, order, c.scale, y=want)
        torch.cuda.synchronize()
    y, now = c.y.clone(), ids[0].clone()

    def step(i):
        now.copy_(ids[i % 4])
        order = lora.adapter_order(now, 5)
        lora.lora_add(c.x, c.a, c.b, order, c.scale, y=y, out=y)

    for i in range(24):
        step(i)
    assert torch.equal(y, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for i in range(4):
            step(i)
    for _ in range(3):
        y.copy_(c.y)
        for _ in range(6):
            g.replay()
        assert torch.equal(y, want)
    # the gradient of one call as the next one's input
    grad, all_of = c.grad, []
    for chained in (False, True):
        gx, sums = torch.zeros_like(c.x), []
        for i in range(8):
            gx, da, db = lora.lora_grad(grad, c.x, c.a, c.b, c.order, c.scale, grad_x=gx, in_place=chained)
            sums += [da, db]
            if not chained:
                torch.cuda.synchronize()
        all_of.append([gx.clone(), *sums])
    assert all(torch.equal(p, q) for p, q in zip(*all_of))


def check_float16_rows(got, want, size, first, second, largest, sizes):
    """As ``check``, for float16 rows of an adapter whose values between the contractions differ widely.  They are
    kept relative to the largest of them, ``largest``, at 2^15: a value's two numbers are off by at most half of
    float16's smallest number each, together 2^-24 of what 2^14 or more stand for, 2^-38 of the largest; the sum over
    the rows by that times the sum of the other factor's ``sizes``."""
    half = torch.finfo(got.dtype).eps / 2
    rel = (first / 16 + 8 + 2 * second / 16 + 8) * 2.0 ** -22 + half * half * 1.01 + 4 * 2.0 ** -24
    slack = size * rel + 2.0 ** -38 * 1.01 * largest * sizes
    tiny = torch.finfo(got.dtype).smallest_normal * torch.finfo(got.dtype).eps / 2
    err = (got.cpu().double() - want).abs()
    bad = ~(err <= slack + half * (want.abs() + slack) + tiny)
    assert not bool(bad.any()), (float(err.max()), float(want.abs().max()), int(bad.sum()), bad.nonzero()[:4].tolist())


def check_float16_weights(c, ranks=slice(None)):
    """The weights' gradients of a float16 case against 64 bits (of the given rank rows and columns)."""
    _, da, db = lora.lora_grad(c.grad, c.x, c.a, c.b, c.order, c.scale)
    _, (wa, sa), (wb, sb) = exact_grad(c.grad, c.x, c.a, c.b, c.ids, c.scale, None)
    m, k, n = c.x.shape[0], c.x.shape[1], c.grad.shape[1]
    x, grad = c.x.cpu().double(), c.grad.cpu().double()
    for i in range(c.a.shape[0]):
        at, s = (c.ids == i).nonzero()[:, 0], float(c.scale[i])
        if not len(at):
            assert not da[i].any() and not db[i].any()
            continue
        back, low = s * grad[at] @ c.b[i].cpu().double(), s * x[at] @ c.a[i].cpu().double().T
        check_float16_rows(da[i][ranks], wa[i][ranks], sa[i][ranks], n, m, float(back[:, ranks].abs().max()),
                           x[at].abs().sum(0)[None])
        check_float16_rows(db[i][:, ranks], wb[i][:, ranks], sb[i][:, ranks], k, m, float(low[:, ranks].abs().max()),
                           grad[at].abs().sum(0)[:, None])


#: rows, k, n, rank, adapters: tiles of 16 rows; a cluster's shares of one adapter; several items per CTA
WEIGHT_PLANS = [(40, 128, 96, 16, 1), (600, 128, 128, 16, 1), (600, 128, 128, 64, 1), (1100, 128, 96, 128, 1),
                (700, 512, 512, 16, 40)]


@pytest.mark.parametrize("plan", WEIGHT_PLANS, ids=str)
@pytest.mark.parametrize("levels", [(1e-2,), (1e-4,), (1e-6,), (1e-2, 1e-4, 1e-6)], ids=str)
@pytest.mark.parametrize("small", ["grad", "x", "both"])
def test_float16_weight_gradients_beside_rows_of_zeros(plan, levels, small):
    """Masked tokens: rows of the gradient and of the input that are zero take nothing from the others."""
    m, k, n, rank, adapters = plan
    c = Case(m, k, n, rank, adapters, "f16", seed=rank + m)
    row = torch.arange(m)
    by = torch.tensor(levels)[row % len(levels)].double()
    of = lambda name: by if small in (name, "both") else torch.ones(m, dtype=torch.float64)
    c.grad = (c.grad.cpu().double() * torch.where(row % 5 == 1, 0.0, of("grad"))[:, None]).half().cuda()
    c.x = (c.x.cpu().double() * torch.where(row % 7 == 2, 0.0, of("x"))[:, None]).half().cuda()
    check_float16_weights(c)


@pytest.mark.parametrize("plan", WEIGHT_PLANS, ids=str)
@pytest.mark.parametrize("apart", [12, 20, 24, 25, 26, 30])
def test_float16_weight_gradients_of_rows_far_apart(plan, apart):
    """Rows whose values between the contractions are 2^apart below the others', and whose other factor carries the
    sum: they lose bits (``check_float16_rows``), not everything."""
    m, k, n, rank, adapters = plan
    for low_of_x in (True, False):
        c = Case(m, k, n, rank, adapters, "f16", bare=0, seed=apart)
        even = (torch.arange(m) % 2 == 0)[:, None]
        up, down = 2.0 ** (apart // 2 - 4), 2.0 ** (apart // 2 - 4 - apart)
        low = torch.where(even, up, down).double()
        other = torch.where(even, 2.0 ** -14, 1.0).double()  # the rows below: their products are the larger ones
        x, grad = (low, other) if low_of_x else (other, low)
        c.x, c.grad = (c.x.cpu().double() * x).half().cuda(), (c.grad.cpu().double() * grad).half().cuda()
        check_float16_weights(c)


@pytest.mark.parametrize("plan", WEIGHT_PLANS, ids=str)
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_float16_weight_gradients_beside_a_rank_that_is_not_finite(plan, value):
    """One rank row of A and column of B with a value that is not finite: the other ranks' gradients keep their bits,
    of small values and of values beyond float16's largest."""
    m, k, n, rank, adapters = plan
    others = [r for r in range(rank) if r != 3]
    for grad_std, b_std, x_std, a_std in ((1e-4, 0.1, 1.0, None), (1e3, 100.0, 1e-5, 0.1), (1e-5, 0.1, 1e3, 100.0)):
        c = Case(m, k, n, rank, adapters, "f16", seed=m, x_std=x_std, a_std=a_std, b_std=b_std, grad_std=grad_std)
        c.a[:, 3, 7], c.b[:, 9, 3] = value, value
        _, da, db = lora.lora_grad(c.grad, c.x, c.a, c.b, c.order, c.scale)
        for i in c.ids.unique().tolist():
            if i >= 0:
                assert not bool(torch.isfinite(da[i, 3]).any() or torch.isfinite(db[i, :, 3]).any())
        check_float16_weights(c, others)


def test_float16_infinities_come_through():
    """A row whose only values between the contractions are infinite, beside rows of ordinary ones."""
    for m in (20, 600):
        c = Case(m, 128, 96, 16, 1, "f16", bare=0)
        c.a[0, :, 40] = 0
        c.a[0, 3, 40] = float("inf")
        c.x[:, 40] = c.x[:, 40].abs() + 0.5
        c.x[5] = 0
        c.x[5, 40] = 1
        c.grad[:, :4] = c.grad[:, :4].abs() + 0.5
        _, _, db = lora.lora_grad(c.grad, c.x, c.a, c.b, c.order, c.scale)
        assert bool((db[0, :4, 3] == float("inf")).all())
        assert bool(torch.isfinite(db[0][:, [r for r in range(16) if r != 3]]).all())
        c.b[0, 2] = 0
        c.b[0, 2, 3] = 1
        out = lora.lora_add(c.x, c.a, c.b, c.order, c.scale, y=c.y)
        assert bool((out[:, 2] == float("inf")).all())


@pytest.mark.parametrize("rows,rank", [(1, 16), (100, 16), (4200, 24)])
def test_columns_of_one_matrix(rows, rank):
    """x1, the addend in the result's place, the gradients and what they are of as columns of one matrix: nothing in
    common.  Columns in common are refused, before anything is written."""
    c = Case(rows, 96, 96, rank, 3, "bf16")
    wide = torch.randn(rows, 320, device="cuda").bfloat16()
    x, y, third = wide[:, :96], wide[:, 96:192], wide[:, 200:296]
    before = wide.clone()
    want = lora.lora_add(x.clone(), c.a, c.b, c.order, c.scale, y=y.clone())
    lora.lora_add(x, c.a, c.b, c.order, c.scale, y=y, out=y)
    assert torch.equal(y, want)
    want = lora.lora_grad(y.clone(), x.clone(), c.a, c.b, c.order, c.scale, grad_x=third.clone())
    got = lora.lora_grad(y, x, c.a, c.b, c.order, c.scale, grad_x=third, in_place=True)
    assert all(torch.equal(p, q) for p, q in zip(got, want))
    assert torch.equal(wide[:, :96], before[:, :96]) and torch.equal(wide[:, 296:], before[:, 296:])
    now = wide.clone()
    with pytest.raises(W.WqmmError, match="shares memory"):
        lora.lora_add(x, c.a, c.b, c.order, c.scale, out=wide[:, 88:184])
    with pytest.raises(W.WqmmError, match="shares memory"):
        lora.lora_grad(y, x, c.a, c.b, c.order, c.scale, grad_x=wide[:, 184:280], in_place=True)
    assert torch.equal(wide, now)


def test_raw_handle_of_the_default_stream():
    """Its handle is 0: the call runs there, behind what is already on it."""
    c = Case(300, 256, 128, 16, 3, "bf16")
    want = lora.lora_add(c.x, c.a, c.b, c.order, c.scale, y=c.y)
    assert torch.cuda.default_stream().cuda_stream == 0
    with W._on_stream(0, c.x.get_device()):
        assert torch.cuda.current_stream() == torch.cuda.default_stream()
    y = torch.zeros_like(c.y)
    torch.cuda._sleep(100_000_000)  # 50 ms
    y.copy_(c.y)
    got = lora.lora_add(c.x, c.a, c.b, c.order, c.scale, y=y, stream=0)
    assert torch.equal(got, want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):  # the handle names the stream, whichever is current
        got = lora.lora_add(c.x, c.a, c.b, c.order, c.scale, y=y, stream=0)
    torch.cuda.synchronize()
    assert torch.equal(got, want)


def test_order_of_indexes_that_are_copied_first():
    """One index per request, for its rows: not contiguous, so the call makes a copy, on the given stream too."""
    old, new = torch.zeros(30, 1, dtype=torch.int32, device="cuda"), torch.arange(30, dtype=torch.int32, device="cuda")[:, None]
    ids = old.clone()
    side = torch.cuda.Stream()
    lora.adapter_order(ids.expand(30, 17), 30, stream=side)  # the kernels are loaded: nothing else waits below
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(100_000_000)  # 50 ms
        ids.copy_(new)
    got = lora.adapter_order(ids.expand(30, 17), 30, stream=side)
    side.synchronize()
    want = lora.adapter_order(new.expand(30, 17).reshape(-1), 30)
    assert all(torch.equal(p, q) for p, q in zip(got, want))


def test_projection_refuses_before_it_writes():
    m, k = 40, 128
    c = Case(m, k, k, 16, 4, "bf16")
    q = torch.randint(-128, 128, (k, k), dtype=torch.int8, generator=torch.Generator().manual_seed(1)).cuda()
    s = torch.full((k,), 0.002, dtype=torch.bfloat16, device="cuda")
    out = torch.full_like(c.y, 3)
    half = TokenOrder(c.order.offsets, c.order.source[:m // 2], None)
    for args in ((c.a.float(), c.b, c.order), (c.a[:, :12], c.b, c.order), (c.a, c.b[:2], c.order), (c.a, c.b, half),
                 (c.a.cpu(), c.b, c.order), (c.a, c.b, c.order, c.scale.cpu())):
        with pytest.raises((W.WqmmError, ValueError)):
            lora.lora_weight_quant_matmul(c.x, W.desc(q), s, *args, out=out)
        assert bool((out == 3).all())
    # the adapters read x1 after the projection has written its result
    x = c.x.clone()
    with pytest.raises(ValueError, match="shares memory"):
        lora.lora_weight_quant_matmul(x, W.desc(q), s, c.a, c.b, c.order, out=x)
    assert torch.equal(x, c.x)
    got = lora.lora_weight_quant_matmul(c.x, W.desc(q), s, c.a, c.b, c.order, c.scale, out=out)
    assert got is out and torch.equal(out, lora.lora_weight_quant_matmul(c.x, W.desc(q), s, c.a, c.b, c.order, c.scale))
