"""Layer norm and RMS norm on the GPU against their definitions in 64 bits."""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - CPU container
    pytest.skip("no GPU", allow_module_level=True)

from learned_optimizer_step_amd import layers  # noqa: E402
from learned_optimizer_step_amd import lopt as L  # noqa: E402
from ops_cases import (CODE, TINY, TYPES, U, close, depth, norm_backward, norm_forward, norm_forward_tols,  # noqa: E402
                       rounding, row_depth)

# one row to thousands; every row layout with its first and last width, widths that no vector divides, and rows too long
# for registers
SHAPES = [(1, 1), (3, 2), (1, 768), (5, 7), (1000, 8), (67, 64), (130, 65), (33, 197), (9, 512), (6, 513), (2049, 768),
          (70, 1000), (5, 1024), (7, 1025), (300, 2048), (4, 2049), (3, 4096), (5, 4099), (3, 8192), (2, 8193), (3, 16384),
          (2, 16385), (5, 40001), (9000, 24)]


def make(rows, cols, t, wt, seed, bias=True):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(rows, cols, generator=g) * (0.5 + torch.rand(rows, 1, generator=g)) + torch.randn(1, cols, generator=g))
    dy = torch.randn(rows, cols, generator=g) * 0.1
    w = (1 + 0.2 * torch.randn(cols, generator=g)).to(wt)
    b = (0.2 * torch.randn(cols, generator=g)).to(wt) if bias else None
    return x.to(t), dy.to(t), w, b


def gpu(*ts):
    return [None if v is None else v.cuda() for v in ts]


def check(x, dy, w, b, eps, rms, what):
    t, wt = x.dtype, torch.float32 if w is None else w.dtype
    gx, gdy, gw, gb = gpu(x, dy, w, b)
    y, mean, rstd = layers.norm_forward(gx, gw, gb, eps, rms=rms)
    want = norm_forward(x, w, b, eps, rms)
    ty, tm, tr = norm_forward_tols(*want, t, x)
    close(y, want[0], ty, f"{what} y")
    close(rstd, want[2], tr, f"{what} rstd")
    assert (mean is None) == rms
    if not rms:
        close(mean, want[1], tm[:], f"{what} mean")
    dx, dw, db = layers.norm_backward(gdy, gx, gw, mean, rstd, rms=rms)
    dxe, dwe, dbe, tol, dwa, dba = norm_backward(dy, x, w, None if rms else mean.cpu(), rstd.cpu(), rms)
    close(dx, dxe, rounding(dxe, t) + tol, f"{what} dx")
    k = row_depth(x.shape[0]) * U
    close(dw, dwe, rounding(dwe, wt) + k * dwa, f"{what} dw")
    if rms:
        assert db is None
    else:
        close(db, dbe, rounding(dbe, wt) + k * dba, f"{what} db")


@pytest.mark.parametrize("rms", [False, True], ids=["layer", "rms"])
@pytest.mark.parametrize("t", TYPES, ids=str)
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_against_the_definition(rows, cols, t, rms):
    if not rms and cols == 1:
        eps = 1e-2
    else:
        eps = 1e-5
    # parameters are fp32 as the optimizer's, or of the activations' type
    wt = torch.float32 if (rows + cols) % 2 else t
    check(*make(rows, cols, t, wt, rows * 7 + cols, bias=not rms), eps, rms, f"{rows}x{cols}")


@pytest.mark.parametrize("rms", [False, True], ids=["layer", "rms"])
def test_without_weight_or_bias(rms):
    x, dy, w, b = make(40, 300, torch.bfloat16, torch.float32, 3, bias=not rms)
    check(x, dy, None, None, 1e-6, rms, "neither")
    check(x, dy, w, None, 1e-6, rms, "weight")
    if not rms:
        check(x, dy, None, b, 1e-6, rms, "bias")


def test_rows_far_from_zero_and_without_spread():
    # a mean of 1000 spreads: the fp32 mean alone would be off by 2^-14 spreads
    g = torch.Generator().manual_seed(5)
    x = 1000.0 + torch.randn(50, 768, generator=g)
    check(x, torch.randn(50, 768, generator=g), torch.ones(768), torch.zeros(768), 1e-5, False, "offset")
    # equal values: the output is the bias, but for what rounding leaves of the spread: 2^-24 of 2^-22, times 1 / sqrt(eps)
    x = torch.full((4, 1000), 3.25)
    b = torch.randn(1000, generator=g)
    y, mean, rstd = layers.norm_forward(x.cuda(), torch.ones(1000).cuda(), b.cuda(), 1e-5)
    assert bool(((y.cpu() - b).abs() <= 2.0 ** -46 * 1e3 + U * b.abs()).all()) and torch.equal(mean.cpu(), torch.full((4,), 3.25))
    # zeros through an RMS norm
    y, _, rstd = layers.norm_forward(torch.zeros(3, 70).cuda(), None, None, 1e-6, rms=True)
    assert not y.any() and torch.allclose(rstd.cpu(), torch.full((3,), 1e3), rtol=1e-6)


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_a_row_with_nan_or_infinity_spoils_no_other(bad):
    for cols in (60, 500, 1001, 3000, 9000, 20000):
        x, dy, w, b = make(9, cols, torch.float32, torch.float32, cols)
        good, *_ = layers.norm_forward(*gpu(x, w, b))
        x[4, cols // 2] = bad
        for rms in (False, True):
            y, mean, rstd = layers.norm_forward(*gpu(x, w), None, rms=rms)
            ok = torch.isfinite(y).all(1).cpu()
            assert ok.tolist() == [r != 4 for r in range(9)], (cols, rms)
            if not rms:
                assert torch.isnan(y[4]).all()
            dx = layers.norm_backward(dy.cuda(), x.cuda(), w.cuda(), mean, rstd, rms=rms)[0]
            assert torch.isfinite(dx).all(1).cpu().tolist() == ok.tolist()
        y, *_ = layers.norm_forward(*gpu(x, w, b))
        assert torch.equal(y[:4], good[:4]) and torch.equal(y[5:], good[5:])


def test_strided_rows_and_rows_behind_the_last():
    """x and dy as slices of wider tensors, outputs with a row stride through the library's call: what lies between and
    behind the rows is left as it was."""
    rows, cols, ld = 37, 193, 260
    g = torch.Generator().manual_seed(8)
    for t in TYPES:
        big = torch.randn(rows + 2, ld, generator=g).to(t).cuda()
        x, dy = big[:rows, 3:3 + cols], big[1:rows + 1, 41:41 + cols]
        w, b = torch.randn(cols, generator=g).cuda(), torch.randn(cols, generator=g).cuda()
        y0, mean0, rstd0 = layers.norm_forward(x.contiguous(), w, b)
        y1, mean1, rstd1 = layers.norm_forward(x, w, b)
        assert torch.equal(y0, y1) and torch.equal(mean0, mean1) and torch.equal(rstd0, rstd1)
        want = layers.norm_backward(dy.contiguous(), x.contiguous(), w, mean0, rstd0)
        got = layers.norm_backward(dy, x, w, mean0, rstd0)
        assert all(torch.equal(p, q) for p, q in zip(want, got))
        outs = [torch.full((rows + 2, ld), 7.0, dtype=t, device="cuda") for _ in range(2)]
        stream = torch.cuda.current_stream().cuda_stream
        code, size = CODE[t], outs[0].element_size()
        L.lopt_norm_forward(0, rows, cols, code, x.data_ptr(), ld, w.data_ptr(), b.data_ptr(), 0, 1e-5,
                            outs[0].data_ptr() + 5 * size, ld, None, None, stream)
        L.lopt_norm_backward(0, rows, cols, code, dy.data_ptr(), ld, x.data_ptr(), ld, w.data_ptr(), 0, mean0.data_ptr(),
                             rstd0.data_ptr(), outs[1].data_ptr() + 5 * size, ld, None, None, 0, 0, None, 0, stream)
        for out, ref in zip(outs, (y0, want[0])):
            assert torch.equal(out[:rows, 5:5 + cols], ref)
            out[:rows, 5:5 + cols] = 7.0
            assert bool((out == 7.0).all())


def test_accumulating_and_leaving_out():
    x, dy, w, b = gpu(*make(500, 321, torch.bfloat16, torch.float32, 11))
    _, mean, rstd = layers.norm_forward(x, w, b)
    dx, dw, db = layers.norm_backward(dy, x, w, mean, rstd)
    again = layers.norm_backward(dy, x, w, mean, rstd)
    assert all(torch.equal(p, q) for p, q in zip((dx, dw, db), again)), "the same inputs give the same bits"
    base = torch.randn(2, 321, device="cuda")
    gw, gb = base[0].clone(), base[1].clone()
    layers.norm_backward(dy, x, w, mean, rstd, grad_weight=gw, grad_bias=gb, accumulate=True)
    assert torch.equal(gw, base[0] + dw) and torch.equal(gb, base[1] + db)
    only = layers.norm_backward(dy, x, w, mean, rstd, need_x=False, need_bias=False)
    assert only[0] is None and only[2] is None and torch.equal(only[1], dw)
    only = layers.norm_backward(dy, x, w, mean, rstd, need_x=False, need_weight=False)
    assert only[1] is None and torch.equal(only[2], db)
    only = layers.norm_backward(dy, x, w, mean, rstd, need_weight=False, need_bias=False)
    assert only[1] is None and torch.equal(only[0], dx)


def test_no_rows():
    x = torch.empty(0, 50, device="cuda")
    w = torch.ones(50, device="cuda")
    y, mean, rstd = layers.norm_forward(x, w, w)
    assert y.shape == (0, 50) and rstd.shape == (0,)
    dx, dw, db = layers.norm_backward(x, x, w, mean, rstd)
    assert dx.shape == (0, 50) and not dw.any() and not db.any()
    gw = torch.full((50,), 2.0, device="cuda")
    layers.norm_backward(x, x, w, mean, rstd, grad_weight=gw, need_bias=False, accumulate=True)
    assert bool((gw == 2.0).all())


@pytest.mark.parametrize("rms", [False, True], ids=["layer", "rms"])
def test_autograd_and_differences(rms):
    """Gradients through autograd against central differences of the definition in 64 bits, in random directions."""
    x, dy, w, b = make(12, 90, torch.float32, torch.float32, 21, bias=not rms)
    x = x.view(3, 4, 90)
    leaves = [v.cuda().requires_grad_(True) for v in (x, w) + (() if rms else (b,))]
    y = layers.rms_norm(*leaves, 1e-5) if rms else layers.layer_norm(*leaves, 1e-5)
    assert y.shape == x.shape
    grads = torch.autograd.grad(y, leaves, dy.view(3, 4, 90).cuda())

    def f(x, w, b):
        return (norm_forward(x.reshape(12, 90), w, b, 1e-5, rms)[0] * dy.double()).sum()

    g = torch.Generator().manual_seed(2)
    args = [x.double(), w.double(), None if rms else b.double()]
    for k, grad in enumerate(grads):
        d = torch.randn(args[k].shape, generator=g, dtype=torch.float64)
        h = 1e-4
        plus = f(*[v if j != k else v + h * d for j, v in enumerate(args)])
        minus = f(*[v if j != k else v - h * d for j, v in enumerate(args)])
        want = (plus - minus) / (2 * h)
        got = (grad.double().cpu() * d).sum()
        # differences: h^2 of the third derivative (about the value's size here), and 2^-52 / h; the gradient: its roundings
        tol = 1e-6 * abs(want) + 100 * U * (grad.double().cpu() * d).abs().sum() + 1e-7 * (1 + dy.double().abs().sum())
        assert abs(got - want) <= tol, (k, got, want)


def test_gradients_cannot_be_differentiated():
    x, dy, w, b = gpu(*make(5, 64, torch.float32, torch.float32, 4))
    x.requires_grad_(True)
    grad, = torch.autograd.grad(layers.layer_norm(x, w, b), x, dy, create_graph=True)
    assert torch.equal(grad, torch.autograd.grad(layers.layer_norm(x, w, b), x, dy)[0])
    with pytest.raises(RuntimeError, match="cannot be differentiated"):
        grad.sum().backward()


def test_gradients_that_come_expanded():
    x, dy, w, b = gpu(*make(30, 100, torch.float32, torch.float32, 4))
    x.requires_grad_(True)
    layers.layer_norm(x, w, b).sum().backward()   # dy: one value, expanded with strides of zero
    want = layers.norm_backward(torch.ones_like(x), x.detach(), w, *layers.norm_forward(x.detach(), w, b)[1:])[0]
    assert torch.equal(x.grad, want)


def test_on_another_stream_and_in_a_graph():
    x, dy, w, b = gpu(*make(700, 768, torch.bfloat16, torch.float32, 31))
    want = layers.norm_forward(x, w, b)
    grads = layers.norm_backward(dy, x, w, want[1], want[2])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = layers.norm_forward(x, w, b)
        got_grads = layers.norm_backward(dy, x, w, got[1], got[2])
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(p, q) for p, q in zip(want + grads, got + got_grads))

    xs, gw, gb = x.clone(), torch.zeros(768, device="cuda"), torch.zeros(768, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, mean, rstd = layers.norm_forward(xs, w, b)
        dx, _, _ = layers.norm_backward(dy, xs, w, mean, rstd, grad_weight=gw, grad_bias=gb)
    for k in range(4):
        xs.copy_(x * (1 + k))
        eager = layers.norm_forward(xs, w, b)
        eager_grads = layers.norm_backward(dy, xs, w, eager[1], eager[2])
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(eager + eager_grads, (y, mean, rstd, dx, gw, gb))), k


@pytest.mark.parametrize("rms", [False, True], ids=["layer", "rms"])
@pytest.mark.parametrize("t,rows,cols", [(torch.float32, 50001, 1029), (torch.bfloat16, 13000, 8200)])
def test_gradients_too_large_for_the_caches(t, rows, cols, rms):
    """Over 200 MB the gradient is written another way; the last rows against the same rows alone."""
    x, dy = torch.randn(rows, cols, device="cuda").to(t), torch.randn(rows, cols, device="cuda").to(t)
    w = torch.randn(cols, device="cuda")
    _, mean, rstd = layers.norm_forward(x, w, None, rms=rms)
    dx, dw, db = layers.norm_backward(dy, x, w, mean, rstd, rms=rms)
    for part in (slice(0, 90), slice(rows - 90, rows)):
        m = None if rms else mean[part].clone()
        want = layers.norm_backward(dy[part].clone(), x[part].clone(), w, m, rstd[part].clone(), rms=rms)[0]
        assert torch.equal(dx[part], want)
    xh = (x.double() - (0 if rms else mean.double()[:, None])) * rstd.double()[:, None]
    terms = dy.double() * xh
    # at most rows / 512 + 100 additions of a term
    assert bool(((dw.double() - terms.sum(0)).abs() <= (rows // 512 + 100) * U * terms.abs().sum(0)).all())
    if not rms:
        assert bool(((db.double() - dy.double().sum(0)).abs() <= (rows // 512 + 100) * U * dy.double().abs().sum(0)).all())


def test_more_elements_than_32_bits_count():
    """2^31 + elements (8.6 GB in, 8.6 GB out in bf16): the last rows against the same rows alone."""
    cols, rows = 2048, (1 << 20) + 3
    x = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda")
    x[-70:] = torch.randn(70, cols, device="cuda")
    x[:-70] = 1.0
    w = torch.randn(cols, device="cuda")
    y, mean, rstd = layers.norm_forward(x, w, w)
    part = layers.norm_forward(x[-70:].clone(), w, w)
    assert torch.equal(y[-70:], part[0]) and torch.equal(rstd[-70:], part[2])
    dy = torch.zeros_like(x)
    dy[-70:] = torch.randn(70, cols, device="cuda")
    dx, dw, db = layers.norm_backward(dy, x, w, mean, rstd)
    want = layers.norm_backward(dy[-70:].clone(), x[-70:].clone(), w, part[1], part[2])
    assert torch.equal(dx[-70:], want[0])
    size = dy[-70:].double().abs().sum(0)
    assert bool(((db.double() - want[2].double()).abs() <= 200 * U * size).all())
    assert bool(((dw.double() - want[1].double()).abs() <= 200 * U * 6 * size).all())


def test_refusals_of_the_tensors():
    x, w = torch.ones(4, 8, device="cuda"), torch.ones(8, device="cuda")
    _, mean, rstd = layers.norm_forward(x, w, w)
    for call in (lambda: layers.norm_forward(x, w[:4]), lambda: layers.norm_forward(x, w.cpu()),
                 lambda: layers.norm_forward(x, w, w.bfloat16()), lambda: layers.norm_forward(x.double(), w),
                 lambda: layers.norm_forward(x, w, w, rms=True), lambda: layers.norm_forward(x[0, 0], w),
                 lambda: layers.norm_backward(x.half(), x, w, mean, rstd), lambda: layers.norm_backward(x[:2], x, w, mean, rstd),
                 lambda: layers.norm_backward(x, x, w, None, rstd), lambda: layers.norm_backward(x, x, w, mean, rstd[:3]),
                 lambda: layers.norm_backward(x, x, w, mean, rstd, accumulate=True),
                 lambda: layers.norm_backward(x, x, w, mean, rstd, grad_weight=torch.ones(7, device="cuda"))):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(L.LoptError):
        layers.norm_forward(x, w, w, eps=-1.0)


@pytest.mark.parametrize("rms", [False, True], ids=["layer", "rms"])
def test_weights_of_more_columns_than_one_grid_has_threads_for(rms):
    """The blocks' sums are joined by 32 threads a column: 2^32 threads and more from 2^26 columns (RMS: 2^27) on."""
    rows, cols = 2, (1 << (27 if rms else 26)) + 3
    g = torch.Generator(device="cuda").manual_seed(12)
    x, dy = (torch.randn(rows, cols, generator=g, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    mean = None if rms else torch.tensor([0.25, -0.5], device="cuda")
    rstd = torch.tensor([1.5, 0.75], device="cuda")
    dx, dw, db = layers.norm_backward(dy, x, None, mean, rstd, rms=rms, need_x=False)
    assert dx is None
    for a in range(0, cols, 1 << 24):
        part = slice(a, min(cols, a + (1 << 24)))
        xh = (x[:, part].double() - (0 if rms else mean.double()[:, None])) * rstd.double()[:, None]
        terms = dy[:, part].double() * xh
        # two roundings of xh, one of each product's sum and of the join's
        assert bool(((dw[part].double() - terms.sum(0)).abs() <= 4 * U * terms.abs().sum(0) + TINY[torch.float32]).all()), a
        if not rms:
            d = dy[:, part].double()
            assert bool(((db[part].double() - d.sum(0)).abs() <= U * d.abs().sum(0)).all()), a


def test_the_mean_is_rounded_once():
    """fp32 rows whose mean cancels: the sum is taken in 64 bits, so its error is that of the last rounding (an fp32 sum's
    would be of the size of the values).  A term passes at most `depth` additions in 64 bits."""
    g = torch.Generator().manual_seed(40)
    for cols in (7, 60, 200, 768, 1025, 5000, 16385, 40001):
        x = 100 * torch.randn(40, cols, generator=g)
        x[:, cols // 2] -= x.double().sum(1).float()
        _, mean, _ = layers.norm_forward(x.cuda())
        exact = x.double().mean(1)
        size = x.double().abs().mean(1)
        assert bool((exact.abs() < 1e-5 * size).all())
        close(mean, exact, U * exact.abs() + (depth(cols) + 2) * 2.0 ** -53 * size + TINY[torch.float32], f"{cols} mean")


def test_the_mean_square_of_ones_is_one():
    """The sum of n ones is n and n / n is 1, for every width: the root and its reciprocal too."""
    for cols in (1, 3, 41, 47, 55, 61, 82, 83, 94, 97, 107, 197, 500, 768, 1000, 1003, 2047, 3001, 6000, 16383, 16385, 40001):
        for t in TYPES:
            y, _, rstd = layers.norm_forward(torch.ones(3, cols, dtype=t).cuda(), eps=0.0, rms=True)
            assert bool((rstd == 1).all()) and bool((y == 1).all()), (cols, t)


@pytest.mark.parametrize("cols", [41, 300, 1000, 5000, 20000])
def test_rows_whose_squares_overflow(cols):
    """The sum of squares is a float: above it rstd is 0, as that of an infinity, and no other row is touched."""
    x = torch.ones(3, cols)
    x[1] *= 3e19
    x[1, ::2] *= -1
    for rms in (False, True):
        y, _, rstd = layers.norm_forward(x.cuda(), None, None, 1e-6, rms=rms)
        assert rstd[1] == 0 and not y[1].any()
        assert torch.isfinite(y).all() and (rstd[0::2] > 0).all()


@pytest.mark.parametrize("given,which", [(g, w) for g in ("x", "xw", "xb", "xwb") for w in ("x", "w", "b", "xw", "xb", "wb", "xwb")
                                         if set(w) <= set(g)])
def test_autograd_of_any_of_the_tensors(given, which):
    """Each gradient reaches its own tensor, whichever are there and whichever want one."""
    x, dy, w, b = gpu(*make(20, 130, torch.float32, torch.float32, 51))
    have = {"x": x, "w": w if "w" in given else None, "b": b if "b" in given else None}
    for k in which:
        have[k].requires_grad_(True)
    y = layers.layer_norm(have["x"], have["w"], have["b"])
    got = torch.autograd.grad(y, [have[k] for k in which], dy)
    plain = {k: None if v is None else v.detach() for k, v in have.items()}
    _, mean, rstd = layers.norm_forward(plain["x"], plain["w"], plain["b"])
    want = dict(zip("xwb", layers.norm_backward(dy, plain["x"], plain["w"], mean, rstd)))
    assert all(torch.equal(g, want[k]) for g, k in zip(got, which))
