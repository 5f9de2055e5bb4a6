"""The distillation loss on the GPU against its definition in 64 bits."""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - CPU container
    pytest.skip("no GPU", allow_module_level=True)

from learned_optimizer_step_amd import layers  # noqa: E402
from learned_optimizer_step_amd import lopt as L  # noqa: E402
from ops_cases import CODE, TINY, TYPES, U, close, distill, rounding  # noqa: E402

# (rows, vocabulary, entries, temperature)
SHAPES = [(1, 1, 1, 1.0), (1, 2, 2, 2.0), (3, 7, 3, 0.5), (5, 64, 1, 1.0), (4, 513, 20, 2.0), (300, 1000, 8, 2.0),
          (2, 1001, 300, 1.0), (7, 4097, 33, 4.0), (2, 8191, 65, 0.7), (3, 8192, 1024, 1.0), (2, 50257, 32, 2.0),
          (1, 130001, 100, 1.0), (600, 300, 5, 3.0),
          # every block size, with one and with more entries a thread
          (2100, 900, 70, 1.0), (1100, 2100, 200, 1.0), (1030, 2500, 9, 2.0), (600, 8200, 300, 1.0), (520, 9001, 12, 0.5)]


def make(rows, cols, top, t, ut, idt, seed, absent=0.2):
    g = torch.Generator().manual_seed(seed)
    z = 3 * torch.randn(rows, cols, generator=g)
    u, ids = torch.topk(z + torch.randn(rows, cols, generator=g), top, dim=1)
    u, z = u.to(ut), z.to(t)
    gone = torch.rand(rows, top, generator=g) < absent
    ids[gone] = torch.tensor([-1, -9, cols, cols + 77])[torch.randint(0, 4, (int(gone.sum()),), generator=g)]
    if rows > 2:
        ids[1] = -1
    return z, ids.to(idt), u, torch.randn(rows, generator=g) * 0.3


def tols(z, loss, lse, qp, q, dense, size, terms, tau, t):
    """Each exponent is off by a few U of its size (a product, a sum and the rounding of 1 / tau), the sum of the softmax by
    its additions (vocabulary / 4096 in a thread, 16, 6 and 8 over it, the wave and the block) and by U per exponential."""
    add = z.shape[1] // 4096 + 16 + 40
    e = (8 * size + add) * U
    # every term of the loss: its three parts' roundings, and p's own, of the size of its exponent
    return tau * tau * (e + 16 * U * size + 16 * U * size * terms) + TINY[torch.float32], e


def check(z, ids, u, dl, tau, what):
    t = z.dtype
    loss, lse = layers.distill_forward(z.cuda(), ids.cuda(), u.cuda(), tau)
    dz = layers.distill_backward(dl.cuda(), z.cuda(), ids.cuda(), u.cuda(), lse, tau)
    tau32 = torch.tensor(tau, dtype=torch.float32).double().item()
    want = distill(z, ids, u, tau32)
    tl, e = tols(z, *want, tau32, t)
    close(lse, want[1], e, f"{what} lse")
    close(loss, want[0], tl, f"{what} loss")
    # the gradient with the lse as the forward pass kept it
    _, _, qp, q, dense, size, _ = distill(z, ids, u, tau32, lse.cpu())
    g = (dl.double() * tau32)[:, None]
    tol = g.abs() * U * (8 * size[:, None] * q + (16 * size[:, None] + ids.shape[1]) * dense)
    close(dz, qp * g, rounding(qp * g, t) + tol + g.abs() * 2.0 ** -125, f"{what} dz")
    return loss, lse, dz


@pytest.mark.parametrize("t", TYPES, ids=str)
@pytest.mark.parametrize("rows,cols,top,tau", SHAPES)
def test_against_the_definition(rows, cols, top, tau, t):
    for ut, idt, absent in ((torch.float32, torch.int64, 0.2), (t, torch.int32, 0.0)):
        z, ids, u, dl = make(rows, cols, top, t, ut, idt, rows + cols, absent)
        check(z, ids, u, dl, tau, f"{rows}x{cols} top {top}")


def test_rows_without_entries_and_absent_ones_whatever_they_hold():
    z, ids, u, dl = make(12, 900, 10, torch.float32, torch.float32, torch.int64, 3, absent=0.3)
    loss, lse, dz = check(z, ids, u, dl, 2.0, "plain")
    u2 = u.clone()
    u2[(ids < 0) | (ids >= 900)] = torch.tensor([math.nan, math.inf, -math.inf, 3e38]).repeat(60)[:int(((ids < 0) | (ids >= 900)).sum())]
    again = check(z, ids, u2, dl, 2.0, "absent")
    assert all(torch.equal(a, b) for a, b in zip((loss, lse, dz), again))
    # entries of -inf are absent, in part or all of a row's
    u3 = u.clone()
    u3[3, ::2] = -math.inf
    u3[4] = -math.inf
    loss, _, dz = check(z, ids, u3, dl, 2.0, "-inf")
    assert loss[4] == 0 and not dz[4].any() and loss[1] == 0 and not dz[1].any()
    # a row without entries has no loss whatever its logits and its share of the gradient are
    z4 = z.clone()
    z4[1, 5], z4[4, 7] = math.nan, math.inf
    loss, lse, dz = (v.cpu() for v in (*layers.distill_forward(z4.cuda(), ids.cuda(), u3.cuda(), 2.0),
                                       layers.distill_backward(dl.cuda(), z4.cuda(), ids.cuda(), u3.cuda(), lse, 2.0)))
    assert loss[1] == 0 and loss[4] == 0 and not dz[1].any() and not dz[4].any()
    assert torch.isnan(lse[1])


def test_an_id_that_is_listed_twice():
    z, ids, u, dl = make(6, 500, 12, torch.float32, torch.float32, torch.int64, 5, absent=0.0)
    ids[:, 5] = ids[:, 0]
    ids[:, 11] = ids[:, 0]
    ids[2] = 7                      # every entry the same
    _, _, dz = check(z, ids, u, dl, 1.0, "twice")
    assert torch.equal(dz, check(z, ids, u, dl, 1.0, "again")[2])
    z, ids, u, dl = make(2, 30000, 1024, torch.bfloat16, torch.float32, torch.int32, 6, absent=0.0)
    ids[:, 500:] = ids[:, :524]
    check(z, ids, u, dl, 1.0, "half of the list twice")


def test_masked_logits():
    """A vocabulary masked with -inf, or with the type's lowest value; NaN and +inf spoil their own row."""
    for t in TYPES:
        z, ids, u, dl = make(8, 3000, 16, t, torch.float32, torch.int64, 7, absent=0.0)
        keep = torch.zeros_like(z, dtype=torch.bool).scatter_(1, ids.clamp(min=0), True)
        for low in (-math.inf, torch.finfo(t).min):
            m = torch.where(keep | (torch.arange(3000) % 3 == 0), z, torch.tensor(low).to(t))
            check(m, ids, u, dl, 2.0, f"{t} {low}")
        m = torch.where(keep & (torch.arange(3000) != ids[0, 0]), z, torch.tensor(-math.inf).to(t))
        loss, lse = layers.distill_forward(m.cuda(), ids.cuda(), u.cuda(), 1.0)
        assert loss[0] == math.inf       # the teacher wants what the student excludes
        assert torch.isfinite(lse).all()
        dz = layers.distill_backward(dl.cuda(), m.cuda(), ids.cuda(), u.cuda(), lse, 1.0)
        assert torch.isfinite(dz).all()
        m = z.clone()
        m[3, 9], m[5, 2500], m[6] = math.nan, math.inf, -math.inf
        loss, lse = layers.distill_forward(m.cuda(), ids.cuda(), u.cuda(), 1.0)
        good = [r not in (3, 5, 6) for r in range(8)]
        assert torch.isfinite(loss).tolist() == good and torch.isnan(lse[3]) and lse[6] == -math.inf
        dz = layers.distill_backward(dl.cuda(), m.cuda(), ids.cuda(), u.cuda(), lse, 1.0)
        assert torch.isfinite(dz).all(1).tolist() == good


def test_peaked_and_far_logits():
    z, ids, u, dl = make(6, 2000, 20, torch.float32, torch.float32, torch.int64, 9, absent=0.0)
    check(z * 200, ids, u * 200, dl, 1.0, "peaked")
    check(z + 1e4, ids, u - 1e4, dl, 1.0, "far")
    check(z, ids, u, dl, 1e-3, "cold")
    check(z, ids, u, dl, 1e3, "hot")


def test_strides_in_place_and_what_lies_around():
    rows, cols, top, ld = 21, 777, 9, 801
    for t in TYPES:
        z, ids, u, dl = make(rows, cols, top, t, torch.float32, torch.int64, 10)
        loss, lse, dz = check(z, ids, u, dl, 2.0, "plain")
        big = torch.full((rows + 1, ld), 9.0, dtype=t, device="cuda")
        big[:rows, 4:4 + cols] = z.cuda()
        wide_i, wide_u = torch.full((rows, 15), 3).cuda(), torch.zeros(rows, 13).cuda()
        wide_i[:, 2:2 + top], wide_u[:, 1:1 + top] = ids.cuda(), u.cuda()
        zs, is_, us = big[:rows, 4:4 + cols], wide_i[:, 2:2 + top], wide_u[:, 1:1 + top]
        l2, s2 = layers.distill_forward(zs, is_, us, 2.0)
        # other addresses, other vectors: the sums may be taken in another order
        assert torch.allclose(loss, l2, rtol=1e-4, atol=1e-5) and torch.allclose(lse, s2, rtol=1e-6)
        stream, code = torch.cuda.current_stream().cuda_stream, CODE[t]
        g = dl.cuda()
        at = big.data_ptr() + 4 * big.element_size()
        L.lopt_distill_backward(rows, cols, code, g.data_ptr(), 1, at, ld, top, is_.data_ptr(), 15, 8, us.data_ptr(), 13, 0, 2.0,
                                lse.data_ptr(), at, ld, stream)      # over the logits
        assert torch.equal(big[:rows, 4:4 + cols], dz)
        big[:rows, 4:4 + cols] = 9.0
        assert bool((big == 9.0).all())
        buf = z.cuda()
        assert layers.distill_backward(g, buf, ids.cuda(), u.cuda(), lse, 2.0, out=buf) is buf and torch.equal(buf, dz)


def test_one_weight_for_all_rows_and_autograd():
    z, ids, u, _ = make(24, 600, 10, torch.float32, torch.float32, torch.int64, 11)
    z3, i3, u3 = z.view(4, 6, 600).cuda().requires_grad_(True), ids.view(4, 6, 10).cuda(), u.view(4, 6, 10).cuda()
    loss = layers.distill_loss(z3, i3, u3, 2.0)
    assert loss.shape == (4, 6)
    grad, = torch.autograd.grad(loss.mean(), z3)      # one value for all rows, expanded
    _, lse = layers.distill_forward(z.cuda(), ids.cuda(), u.cuda(), 2.0)
    want = layers.distill_backward(torch.full((24,), 1 / 24).cuda(), z.cuda(), ids.cuda(), u.cuda(), lse, 2.0)
    assert torch.equal(grad.view(24, 600), want)
    # central differences of the definition in 64 bits
    d = torch.randn(24, 600, generator=torch.Generator().manual_seed(1), dtype=torch.float64)
    h = 1e-4
    diff = (distill(z.double() + h * d, ids, u, 2.0)[0] - distill(z.double() - h * d, ids, u, 2.0)[0]).mean() / (2 * h)
    got = (grad.view(24, 600).double().cpu() * d).sum()
    assert abs(got - diff) <= 1e-6 * abs(diff) + 200 * U * (grad.view(24, 600).double().cpu() * d).abs().sum() + 1e-8


def test_on_another_stream_and_in_a_graph():
    z, ids, u, dl = make(50, 5000, 12, torch.bfloat16, torch.float32, torch.int64, 13)
    z, ids, u, dl = z.cuda(), ids.cuda(), u.cuda(), dl.cuda()
    loss, lse = layers.distill_forward(z, ids, u, 2.0)
    dz = layers.distill_backward(dl, z, ids, u, lse, 2.0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        l2, s2 = layers.distill_forward(z, ids, u, 2.0)
        d2 = layers.distill_backward(dl, z, ids, u, s2, 2.0)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(loss, l2) and torch.equal(lse, s2) and torch.equal(dz, d2)
    zs = z.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        l3, s3 = layers.distill_forward(zs, ids, u, 2.0)
        d3 = layers.distill_backward(dl, zs, ids, u, s3, 2.0)
    for k in range(4):
        zs.copy_(z * (k + 1))
        le, se = layers.distill_forward(zs, ids, u, 2.0)
        de = layers.distill_backward(dl, zs, ids, u, se, 2.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(le, l3) and torch.equal(se, s3) and torch.equal(de, d3), k


def test_no_rows_and_more_elements_than_32_bits_count():
    e = torch.empty(0, 30, device="cuda")
    i, u = torch.empty(0, 4, dtype=torch.int64, device="cuda"), torch.empty(0, 4, device="cuda")
    loss, lse = layers.distill_forward(e, i, u)
    assert loss.shape == (0,) and layers.distill_backward(loss, e, i, u, lse).shape == (0, 30)
    rows, cols = 33000, 65537           # 2^31 + 15 M elements
    z = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    z[-3:] = torch.randn(3, cols, device="cuda")
    ids = torch.randint(0, cols, (rows, 6), device="cuda")
    u = torch.randn(rows, 6, device="cuda")
    loss, lse = layers.distill_forward(z, ids, u)
    # not the bits of a copy of these rows: they begin at other places of a 16-byte piece (65537 elements of 2 bytes a row),
    # so other threads add other elements, and each of the two is off by up to `tols` by itself
    last = z[-3:].cpu(), ids[-3:].cpu(), u[-3:].cpu()
    want = distill(*last, 1.0)
    tl, te = tols(last[0], *want, 1.0, torch.bfloat16)
    close(loss[-3:], want[0], tl, "loss of the last rows")
    close(lse[-3:], want[1], te, "lse of the last rows")
    assert bool(((lse[:-3] - math.log(cols)).abs() <= 60 * U * 12).all())
    g = torch.ones(rows, device="cuda")
    want = layers.distill_backward(g[-3:], z[-3:].clone(), ids[-3:], u[-3:], lse[-3:])
    layers.distill_backward(g, z, ids, u, lse, out=z)
    assert torch.equal(z[-3:], want)


def test_refusals_of_the_tensors():
    z, i, u = torch.ones(3, 8, device="cuda"), torch.zeros(3, 2, dtype=torch.int64, device="cuda"), torch.ones(3, 2, device="cuda")
    loss, lse = layers.distill_forward(z, i, u)
    for call in (lambda: layers.distill_loss(z, i, u[:, :1]), lambda: layers.distill_loss(z, i[:2], u[:2]),
                 lambda: layers.distill_loss(z, i.float(), u), lambda: layers.distill_loss(z, i.cpu(), u),
                 lambda: layers.distill_loss(z.double(), i, u), lambda: layers.distill_backward(loss.half(), z, i, u, lse),
                 lambda: layers.distill_backward(loss, z, i, u, lse[:2]),
                 lambda: layers.distill_backward(loss, z, i, u, lse, out=z.half())):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: layers.distill_loss(z, i, u, 0.0), lambda: layers.distill_loss(z, i, u, float("nan")),
                 lambda: layers.distill_loss(z, i.repeat(1, 600), u.repeat(1, 600))):
        with pytest.raises(L.LoptError):
            call()


def shifted(z, ids, u, tau):
    """The definition with the rows' largest values taken off (in 64 bits, so the bounds do not grow with them): the loss
    and q - p are the same."""
    z, u = z.double(), u.double()
    return distill(z - z.max(1, keepdim=True).values, ids, u - u.max(1, keepdim=True).values, tau)


@pytest.mark.parametrize("tau", [0.25, 1.0])
@pytest.mark.parametrize("t", TYPES, ids=str)
def test_threads_that_see_only_the_lowest_value(t, tau):
    """A vocabulary whose end is masked with the type's lowest value, which overflows when it is scaled: all that most
    threads see of a row.  In 64 bits it is as good as -inf."""
    for cols, kept in ((3000, 700), (9000, 8), (50001, 300)):
        z, ids, u, dl = make(6, cols, 5, t, torch.float32, torch.int64, cols, absent=0.0)
        ids = torch.where(ids < 0, ids, ids % kept)
        z[:, kept:] = torch.finfo(t).min
        loss, lse = layers.distill_forward(z.cuda(), ids.cuda(), u.cuda(), tau)
        dz = layers.distill_backward(dl.cuda(), z.cuda(), ids.cuda(), u.cuda(), lse, tau)
        m = z.clone()
        m[:, kept:] = -math.inf
        want = distill(m, ids, u, tau)
        tl, e = tols(m, *want, tau, t)
        close(lse, want[1], e, f"{cols} lse")
        close(loss, want[0], tl, f"{cols} loss")
        _, _, qp, q, dense, size, _ = distill(m, ids, u, tau, lse.cpu())
        g = (dl.double() * tau)[:, None]
        tol = g.abs() * U * (8 * size[:, None] * q + (16 * size[:, None] + ids.shape[1]) * dense)
        close(dz, qp * g, rounding(qp * g, t) + tol + g.abs() * 2.0 ** -125, f"{cols} dz")


@pytest.mark.parametrize("tau", [0.25, 1.0])
@pytest.mark.parametrize("t", TYPES, ids=str)
def test_rows_of_nothing_but_the_lowest_value(t, tau):
    """The student's distribution is uniform; the gradient cannot be exact (lse holds no log of the count there) but is a
    number, so a mask behind it gives zeros."""
    z, ids, u, dl = make(4, 2500, 9, t, torch.float32, torch.int64, 2, absent=0.0)
    z[2:] = torch.finfo(t).min
    loss, lse = layers.distill_forward(z.cuda(), ids.cuda(), u.cuda(), tau)
    want = shifted(z, ids, u, tau)
    close(loss, want[0], tols(z, *want, tau, t)[0], "loss")
    assert torch.isfinite(lse).all()
    assert torch.isfinite(layers.distill_backward(dl.cuda(), z.cuda(), ids.cuda(), u.cuda(), lse, tau)).all()


@pytest.mark.parametrize("ut", TYPES, ids=str)
def test_teachers_whose_logits_overflow_when_scaled(ut):
    """Lists of nothing but the type's lowest or largest value are lists of equal entries; only -inf is absent."""
    z, ids, u, dl = make(6, 700, 8, torch.float32, ut, torch.int64, 4, absent=0.0)
    u[0], u[2], u[3, 3:] = torch.finfo(ut).min, torch.finfo(ut).max, torch.finfo(ut).min
    u[4] = torch.finfo(ut).min
    u[4, 6:] = -math.inf
    tau = 0.25
    loss, lse = layers.distill_forward(z.cuda(), ids.cuda(), u.cuda(), tau)
    want = shifted(z, ids, u, tau)
    # entries that the teacher excludes have no part in the sizes
    size = torch.where(want[5] > 1e6, 1 + 4 * (z.double() / tau).abs().max(1).values, want[5])
    close(loss, want[0], tols(z, *want[:5], size, want[6], tau, torch.float32)[0], "loss")
    dz = layers.distill_backward(dl.cuda(), z.cuda(), ids.cuda(), u.cuda(), lse, tau)
    u64 = u.double() - u.double().max(1, keepdim=True).values
    _, _, qp, q, dense, size, _ = distill(z, ids, u64, tau, lse.cpu())
    size = torch.where(size > 1e6, 1 + 4 * (z.double() / tau).abs().max(1).values, size)
    g = (dl.double() * tau)[:, None]
    tol = g.abs() * U * (8 * size[:, None] * q + (16 * size[:, None] + 8) * dense)
    close(dz, qp * g, rounding(qp * g, torch.float32) + tol + g.abs() * 2.0 ** -125, "dz")


@pytest.mark.parametrize("tau", [1.0, 3.0, 4.0])
def test_the_offset_of_all_logits_costs_nothing(tau):
    """Student and teacher far from zero, in vocabularies of a few elements and of thousands: the loss has the bound of the
    same logits about zero, 1000 U tau^2 for most of the small ones.  Roundings of the logits scaled by log2 e or 1 / tau,
    half a step of which is 2^-13 (2048 U) or more here, do not keep it."""
    for cols, top in ((3, 2), (7, 7), (40, 5), (5000, 30)):
        z, ids, u, dl = make(64, cols, top, torch.float32, torch.float32, torch.int64, cols, absent=0.0)
        z, u = z + 1e4, u - 1.3e4
        loss, lse = layers.distill_forward(z.cuda(), ids.cuda(), u.cuda(), tau)
        want = shifted(z, ids, u, tau)
        tl, _ = tols(z, *want, tau, torch.float32)
        close(loss, want[0], tl, f"{cols} loss")
        # of lse: the product with the rounded 1 / tau, its own rounding, and the bound about zero
        exact = torch.logsumexp(z.double() / tau, 1)
        close(lse, exact, tols(z, *want, tau, torch.float32)[1] + 3 * U * exact.abs(), f"{cols} lse")
        dz = layers.distill_backward(dl.cuda(), z.cuda(), ids.cuda(), u.cuda(), lse, tau)
        g = (dl.double() * tau)[:, None]
        _, _, qp, q, dense, size, _ = distill(z, ids, u.double() - u.double().max(1, keepdim=True).values, tau, lse.cpu())
        # the student's share has the size of z / tau - lse, two large numbers here; the teacher's has not
        spread = 1 + (u.max(1).values - u.min(1).values).double() / tau
        tol = g.abs() * U * (8 * size[:, None] * q + (16 * spread[:, None] + top) * dense)
        close(dz, qp * g, rounding(qp * g, torch.float32) + tol + g.abs() * 2.0 ** -125, f"{cols} dz")


def test_a_gradient_over_the_logits_is_seen_by_autograd():
    """out=logits is a change in place: a loss that still needs the logits refuses, as after any other."""
    z, ids, u, dl = make(5, 60, 4, torch.float32, torch.float32, torch.int64, 8, absent=0.0)
    z, ids, u, dl = z.cuda(), ids.cuda(), u.cuda(), dl.cuda()
    logits = z.clone().requires_grad_(True) * 1.0
    loss = layers.distill_loss(logits, ids, u)
    _, lse = layers.distill_forward(z, ids, u)
    layers.distill_backward(dl, logits.detach(), ids, u, lse, out=logits.detach())
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.sum().backward()


def test_every_buffer_that_is_written_counts_as_changed():
    x, w = torch.randn(6, 40, device="cuda"), torch.ones(40, device="cuda")
    _, mean, rstd = layers.norm_forward(x, w, w)
    gw, gb, gt = torch.zeros(40, device="cuda"), torch.zeros(40, device="cuda"), torch.zeros(9, 40, device="cuda")
    layers.norm_backward(x, x, w, mean, rstd, grad_weight=gw, grad_bias=gb, accumulate=True)
    layers.embedding_backward(x, torch.arange(6, device="cuda"), 9, out=gt)
    assert [v._version for v in (gw, gb, gt)] == [1, 1, 1]
    with torch.inference_mode():     # has no count, and needs none
        gt = torch.zeros(9, 40, device="cuda")
    layers.embedding_backward(x, torch.arange(6, device="cuda"), 9, out=gt)
    assert torch.equal(gt[:6], x)


def test_one_row_whose_weight_has_a_large_stride():
    """The stride of a dimension of one element means nothing, whatever it is."""
    z, ids, u, dl = make(1, 90, 4, torch.float32, torch.float32, torch.int64, 8, absent=0.0)
    z, ids, u, dl = z.cuda(), ids.cuda(), u.cuda(), dl.cuda()
    _, lse = layers.distill_forward(z, ids, u)
    want = layers.distill_backward(dl, z, ids, u, lse)
    assert torch.equal(layers.distill_backward(dl.as_strided((1,), (1 << 28,)), z, ids, u, lse), want)


@pytest.mark.parametrize("t", TYPES, ids=str)
def test_rows_that_are_read_past_the_cache(t):
    """The first rows of more than 200 MB are read another way than the last ones."""
    cols, rows = 20001, 240_000_000 // (20001 * torch.finfo(t).bits // 8)
    g = torch.Generator(device="cuda").manual_seed(17)
    z = (3 * torch.randn(rows, cols, generator=g, device="cuda")).to(t)
    ids = torch.randint(0, cols, (rows, 12), generator=g, device="cuda")
    u = torch.randn(rows, 12, generator=g, device="cuda")
    dl = torch.randn(rows, generator=g, device="cuda")
    loss, lse = layers.distill_forward(z, ids, u, 2.0)
    dz = layers.distill_backward(dl, z, ids, u, lse, 2.0)
    for part in (slice(0, 24), slice(rows // 6 - 12, rows // 6 + 12), slice(rows - 24, rows)):
        zp, ip, up, lp = (v[part].cpu() for v in (z, ids, u, lse))
        want = distill(zp, ip, up, 2.0)
        tl, e = tols(zp, *want, 2.0, t)
        close(lse[part], want[1], e, f"{part} lse")
        close(loss[part], want[0], tl, f"{part} loss")
        _, _, qp, q, dense, size, _ = distill(zp, ip, up, 2.0, lp)
        s = (dl[part].double().cpu() * 2.0)[:, None]
        tol = s.abs() * U * (8 * size[:, None] * q + (16 * size[:, None] + 12) * dense)
        close(dz[part], qp * s, rounding(qp * s, t) + tol + s.abs() * 2.0 ** -125, f"{part} dz")


def test_strided_logits_within_the_bounds():
    """Rows that begin at other places of a 16-byte piece, each within the bounds by itself."""
    rows, cols, top, ld = 21, 777, 9, 801
    for t in TYPES:
        z, ids, u, dl = make(rows, cols, top, t, torch.float32, torch.int64, 10)
        big = torch.full((rows + 1, ld), 9.0, dtype=t, device="cuda")
        want = distill(z, ids, u, 2.0)
        tl, e = tols(z, *want, 2.0, t)
        for at in (0, 1, 4, 7):
            big[:rows, at:at + cols] = z.cuda()
            loss, lse = layers.distill_forward(big[:rows, at:at + cols], ids.cuda(), u.cuda(), 2.0)
            close(loss, want[0], tl, f"{t} {at} loss")
            close(lse, want[1], e, f"{t} {at} lse")


@pytest.mark.parametrize("tau", [0.25, 1.0, 3.0])
@pytest.mark.parametrize("mask", [-1e6, -1e9, -3e10, -1e20, -1e30])
@pytest.mark.parametrize("t", [torch.float32, torch.bfloat16], ids=str)
def test_masks_of_large_finite_values(t, mask, tau):
    """As good as -inf, in threads that see nothing else too: half a step of the scaled mask is no exponent."""
    for cols, kept in ((3000, 700), (50001, 300)):
        z, ids, u, dl = make(6, cols, 5, t, torch.float32, torch.int64, cols, absent=0.0)
        ids = torch.where(ids < 0, ids, ids % kept)
        g = torch.Generator().manual_seed(cols)
        m, z = z.clone(), z.clone()
        z[:, kept:] = (mask * (1 + torch.rand(6, cols - kept, generator=g))).to(t)
        m[:, kept:] = -math.inf
        loss, lse = layers.distill_forward(z.cuda(), ids.cuda(), u.cuda(), tau)
        want = distill(m, ids, u, tau)
        tl, e = tols(m, *want, tau, t)
        close(lse, want[1], e, f"{cols} lse")
        close(loss, want[0], tl, f"{cols} loss")
        dz = layers.distill_backward(dl.cuda(), z.cuda(), ids.cuda(), u.cuda(), lse, tau)
        _, _, qp, q, dense, size, _ = distill(m, ids, u, tau, lse.cpu())
        s = (dl.double() * tau)[:, None]
        tol = s.abs() * U * (8 * size[:, None] * q + (16 * size[:, None] + 5) * dense)
        close(dz, qp * s, rounding(qp * s, t) + tol + s.abs() * 2.0 ** -125, f"{cols} dz")


@pytest.mark.parametrize("tau", [1e-12, 1e-3, 0.25, 1.0, 3.0])
@pytest.mark.parametrize("at", [-1e30, -3e10, 1e6, 1e10, 1e12])
@pytest.mark.parametrize("t", [torch.float32, torch.bfloat16], ids=str)
def test_rows_far_from_zero(t, at, tau):
    """Rows about a large value: the loss is exact; the gradient is off by the rounding of lse, which can be all of it, but
    no element is larger than the loss's weight times 1 + the teacher's share."""
    z, ids, u, dl = make(4, 2500, 9, torch.float32, torch.float32, torch.int64, 2, absent=0.0)
    z = (z + at).to(t)
    loss, lse = layers.distill_forward(z.cuda(), ids.cuda(), u.cuda(), tau)
    want = shifted(z, ids, u, torch.tensor(tau, dtype=torch.float32).double().item())
    close(loss, want[0], tols(z, *want, tau, t)[0] + 2 * U * want[0].abs(), "loss")
    dz = layers.distill_backward(dl.cuda(), z.cuda(), ids.cuda(), u.cuda(), lse, tau).double().cpu()
    assert bool((dz.abs() <= (1 + 2.0 ** -7) * dl.double().abs()[:, None] * tau).all())


def test_the_coldest_temperatures():
    """Near zero the loss is tau times the largest logit's lead over the taught one, also where tau^2 is no float."""
    z = torch.tensor([[3.0, 1.0, -2.0], [0.0, 5.0, 4.0]])
    ids, u = torch.tensor([[1], [2]]), torch.zeros(2, 1)
    for tau in (1e-6, 1e-20, 1e-25, 1e-30):
        t32 = torch.tensor(tau, dtype=torch.float32).double().item()
        loss, _ = layers.distill_forward(z.cuda(), ids.cuda(), u.cuda(), tau)
        want = t32 * torch.tensor([2.0, 1.0], dtype=torch.float64)
        close(loss, want, 8 * U * want, f"{tau}")     # 1 / tau, its product with the lead, two factors tau, and log s = 0


def test_a_target_is_a_list_of_one_entry():
    """At temperature 1: the cross-entropy of the target, 0 and no gradient where it is an id to ignore."""
    rows, cols = 40, 700
    z, _, _, dl = make(rows, cols, 1, torch.float32, torch.float32, torch.int64, 30)
    target = torch.randint(0, cols, (rows,), generator=torch.Generator().manual_seed(6))
    target[::7] = -100
    leaf = z.cuda().requires_grad_(True)
    loss = layers.distill_loss(leaf, target.cuda()[:, None], torch.zeros(rows, 1, device="cuda"))
    grad, = torch.autograd.grad(loss, leaf, dl.cuda())
    z64 = z.double().requires_grad_(True)
    want = torch.nn.functional.cross_entropy(z64, target, reduction="none", ignore_index=-100)
    want_grad, = torch.autograd.grad(want, z64, dl.double())
    size = 1 + z.double().abs().max(1).values * 2 + 10
    e = (24 * size + 56) * U       # the lse's bound, and the logit's own parts
    close(loss, want.detach(), e * (target >= 0), "loss")
    g = dl.double().abs()[:, None] * (target >= 0)[:, None]
    close(grad, want_grad, g * (e + 2 * U)[:, None], "gradient")
