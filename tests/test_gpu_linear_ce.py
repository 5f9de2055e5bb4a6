"""The cross entropy of a linear layer's logits on the GPU against its definition in 64 bits."""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - CPU container
    pytest.skip("no GPU", allow_module_level=True)

from learned_optimizer_step_amd import layers  # noqa: E402
from learned_optimizer_step_amd import lopt as L  # noqa: E402
from linear_ce_cases import backward, forward  # noqa: E402
from ops_cases import CODE, TYPES, U, close, rounding  # noqa: E402

# (tokens, vocabulary, width): ones, tiles with their neighbours, widths that no stage divides, long vocabularies and many tokens
SIZES = [(1, 1, 1), (1, 2, 8), (3, 1000, 65), (5, 300, 64), (255, 256, 32), (256, 257, 64), (257, 255, 128), (300, 5000, 96), (700, 1025, 333),
         (64, 20000, 200), (1, 30000, 768), (2100, 130, 1024), (513, 769, 2050), (40, 77, 4100)]


def make(n, vocab, dim, t, seed, pad=0.2, gscale=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(n, dim, generator=g)
    w = torch.randn(vocab, dim, generator=g) * (2.5 / math.sqrt(dim))
    targets = torch.randint(0, vocab, (n,), generator=g)
    x = x + 2 * torch.rand(n, 1, generator=g) * w[targets]
    off = torch.rand(n, generator=g)
    targets[off < pad] = -1
    targets[off < pad / 2] = vocab
    targets[off < pad / 4] = -100
    return x.to(t), w.to(t), targets, gscale * (0.5 + torch.rand(n, generator=g)) / n


def check(x, w, targets, g, what, grad_dtype=None, device="cpu"):
    t = x.dtype
    gx, gw, gt, gg = (v.cuda() for v in (x, w, targets, g))
    loss, lse = layers.linear_ce_forward(gx, gw, gt)
    rx, rw, rt, rg = (v.to(device) for v in (x, w, targets, g))
    wl, ws, _, _, tl, ts, there = forward(rx, rw, rt)
    close(loss, wl.cpu(), tl.cpu(), f"{what} loss")
    close(lse, ws.cpu(), ts.cpu(), f"{what} lse")
    assert not loss[~there.to(loss.device)].any()
    dx, dw = layers.linear_ce_backward(gg, gx, gw, gt, lse, grad_dtype=grad_dtype)
    wx, ww, tx, tw = backward(rg, rx, rw, rt)
    assert dx.dtype == t and dw.dtype == (grad_dtype or t)
    close(dx, wx.cpu(), (rounding(wx, t) + tx).cpu(), f"{what} dx")
    close(dw, ww.cpu(), (rounding(ww, dw.dtype) + tw).cpu(), f"{what} dw")
    assert not dx[~there.to(dx.device)].any()


@pytest.mark.parametrize("t", TYPES, ids=str)
@pytest.mark.parametrize("n,vocab,dim", SIZES)
def test_against_the_definition(n, vocab, dim, t):
    scale = 1024.0 if t == torch.float16 else 1.0
    x, w, targets, g = make(n, vocab, dim, t, n + vocab + dim, gscale=scale)
    check(x, w, targets if n % 2 else targets.int(), g, f"{n} of {vocab} x {dim}", grad_dtype=torch.float32 if vocab % 2 else None, device="cuda")


@pytest.mark.parametrize("t,n,vocab,dim", [(torch.bfloat16, 20000, 9000, 64), (torch.float16, 300, 70000, 1024), (torch.float32, 9000, 9001, 96),
                                           (torch.bfloat16, 4000, 30011, 1001)])
def test_vocabularies_in_several_pieces(t, n, vocab, dim):
    """More than 128 MiB of logits, or of a weight that has to be laid out anew."""
    x, w, targets, g = (v.cuda() for v in make(n, vocab, dim, t, 5, gscale=1024.0))
    check(x, w, targets, g, f"{n} of {vocab} x {dim}", device="cuda")


def test_entries_of_minus_infinity():
    """A weight's row of -inf under positive tokens: its logits are -inf, its probabilities and its gradient 0."""
    for t in TYPES:
        x, w, targets, g = make(5, 300, 40, t, 12, pad=0.0)
        x, targets = x.abs() + 0.25, targets.clamp(min=10)
        w[7] = -6e4   # logits so low that nothing is left of them
        want = layers.linear_ce_forward(x.cuda(), w.cuda(), targets.cuda())
        dw = layers.linear_ce_backward(g.cuda(), x.cuda(), w.cuda(), targets.cuda(), want[1], need_x=False)[1]
        w[7] = -math.inf
        got = layers.linear_ce_forward(x.cuda(), w.cuda(), targets.cuda())
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        again = layers.linear_ce_backward(g.cuda(), x.cuda(), w.cuda(), targets.cuda(), got[1], need_x=False)[1]
        assert torch.equal(again, dw) and not again[7].any()


def test_rows_to_ignore_are_not_read():
    """NaN and infinities in rows without a target: loss 0, gradient 0, and nothing of them in dw."""
    for t in TYPES:
        x, w, targets, g = make(300, 500, 130, t, 9, pad=0.4)
        off = (targets < 0) | (targets >= 500)
        clean = layers.linear_ce_forward(x.cuda(), w.cuda(), targets.cuda())
        want = layers.linear_ce_backward(g.cuda(), x.cuda(), w.cuda(), targets.cuda(), clean[1])
        x[off] = math.nan
        x[off.nonzero()[0]] = math.inf
        g[off] = math.nan
        loss, lse = layers.linear_ce_forward(x.cuda(), w.cuda(), targets.cuda())
        assert torch.equal(loss, clean[0]) and torch.equal(lse[~off], clean[1][~off])
        got = layers.linear_ce_backward(g.cuda(), x.cuda(), w.cuda(), targets.cuda(), lse)
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_no_row_has_a_target():
    x, w, _, g = (v.cuda() for v in make(70, 300, 65, torch.bfloat16, 1))
    targets = torch.full((70,), -1, device="cuda")
    loss, lse = layers.linear_ce_forward(x, w, targets)
    dx, dw = layers.linear_ce_backward(g, x, w, targets, lse)
    assert not loss.any() and not dx.any() and not dw.any()
    base = torch.randn(300, 65, device="cuda")
    buf = base.clone()
    layers.linear_ce_backward(g, x, w, targets, lse, grad_weight=buf, accumulate=True)
    assert torch.equal(buf, base)


@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_a_row_with_nan_or_infinity_spoils_no_other_loss(bad):
    for t in TYPES:
        x, w, targets, g = make(40, 700, 64, t, 3, pad=0.0)
        good, lse = layers.linear_ce_forward(x.cuda(), w.cuda(), targets.cuda())
        x[7, 5] = bad
        loss, lse = layers.linear_ce_forward(x.cuda(), w.cuda(), targets.cuda())
        assert torch.isnan(loss[7]) and torch.isnan(lse[7])
        keep = torch.arange(40) != 7
        assert torch.equal(loss[keep], good[keep])
        dx, _ = layers.linear_ce_backward(g.cuda(), x.cuda(), w.cuda(), targets.cuda(), lse)
        assert torch.isnan(dx[7]).all() and torch.isfinite(dx[keep]).all()


def test_entries_of_the_vocabulary_that_are_masked():
    """Weights that drive an entry's logits to -inf or far below take nothing from the others' loss."""
    x = torch.rand(50, 64) + 0.1
    g = torch.Generator().manual_seed(4)
    w = torch.randn(600, 64, generator=g) * 0.3
    targets = torch.randint(100, 600, (50,), generator=g)
    want = torch.nn.functional.cross_entropy(x.double() @ w[100:].double().t(), targets - 100, reduction="none")
    for low in (-math.inf, -1e30, -1e5):
        v = w.clone()
        v[:100] = low
        loss, lse = layers.linear_ce_forward(x.cuda(), v.cuda(), targets.cuda())
        ez = 80 * U * (x.double() @ w[100:].double().abs().t()).max(1).values
        assert bool(((loss.double().cpu() - want).abs() <= 2 * ez + 200 * U * (1 + want)).all()), low
    # a whole tile of them, and a vocabulary of nothing else
    v = torch.full((600, 64), -math.inf)
    v[300] = 0.0
    loss, lse = layers.linear_ce_forward(x.cuda(), v.cuda(), torch.full((50,), 300).cuda())
    assert not loss.any() and not lse.any()


def test_logits_with_a_large_common_offset():
    """Logits around 3000 in bf16: the loss is a difference of them, and keeps its place."""
    g = torch.Generator().manual_seed(6)
    x = torch.cat([torch.randn(60, 64, generator=g), torch.full((60, 64), 8.0)], 1).bfloat16()
    w = torch.cat([torch.randn(2000, 64, generator=g) * 0.3, torch.full((2000, 64), 6.0)], 1).bfloat16()
    targets = torch.randint(0, 2000, (60,), generator=g)
    check(x, w, targets, torch.rand(60, generator=g), "offset")


def test_strides_and_what_lies_around():
    """x and weight as slices of wider tensors (aligned and not), outputs with a row stride: what is around stays."""
    n, vocab, dim = 70, 300, 128
    g = torch.Generator().manual_seed(8)
    for t in TYPES:
        for off, ld in ((0, 256), (16, 160), (3, 197)):
            bx, bw = torch.randn(n + 2, ld, generator=g).to(t).cuda(), (0.2 * torch.randn(vocab + 2, ld, generator=g)).to(t).cuda()
            x, w = bx[1:n + 1, off:off + dim], bw[1:vocab + 1, off:off + dim]
            targets = torch.randint(-1, vocab, (n,), generator=g).cuda()
            gl = torch.rand(n, generator=g).cuda()
            want = layers.linear_ce_forward(x.contiguous(), w.contiguous(), targets)
            got = layers.linear_ce_forward(x, w, targets)
            assert all(torch.equal(a, b) for a, b in zip(want, got))
            grads = layers.linear_ce_backward(gl, x.contiguous(), w.contiguous(), targets, want[1])
            again = layers.linear_ce_backward(gl, x, w, targets, want[1])
            assert all(torch.equal(a, b) for a, b in zip(grads, again))
            ox, ow = (torch.full((r + 2, 211), 7.0, dtype=t, device="cuda") for r in (n, vocab))
            size, code = x.element_size(), CODE[t]
            ws = torch.full((L.lopt_linear_ce_backward_workspace(n, dim, vocab, code) + 256,), 13, dtype=torch.uint8, device="cuda")
            L.lopt_linear_ce_backward(n, dim, vocab, code, gl.data_ptr(), 1, x.data_ptr(), x.stride(0), w.data_ptr(), w.stride(0), targets.data_ptr(), 8,
                                      want[1].data_ptr(), ox.data_ptr() + 5 * size, 211, ow.data_ptr() + 5 * size, 211, code, 0, ws.data_ptr(),
                                      ws.numel() - 256, torch.cuda.current_stream().cuda_stream)
            for out, ref, r in ((ox, grads[0], n), (ow, grads[1], vocab)):
                assert torch.equal(out[:r, 5:5 + dim], ref)
                out[:r, 5:5 + dim] = 7.0
                assert bool((out == 7.0).all())
            assert bool((ws[-256:] == 13).all())


def test_accumulating_leaving_out_and_the_same_bits():
    x, w, targets, g = (v.cuda() for v in make(500, 1500, 321, torch.bfloat16, 11))
    loss, lse = layers.linear_ce_forward(x, w, targets)
    for a, b in zip((loss, lse), layers.linear_ce_forward(x, w, targets)):
        assert torch.equal(a, b)
    dx, dw = layers.linear_ce_backward(g, x, w, targets, lse, grad_dtype=torch.float32)
    for a, b in zip((dx, dw), layers.linear_ce_backward(g, x, w, targets, lse, grad_dtype=torch.float32)):
        assert torch.equal(a, b)
    base = torch.randn(1500, 321, device="cuda")
    buf = base.clone()
    got = layers.linear_ce_backward(g, x, w, targets, lse, grad_weight=buf, accumulate=True, need_x=False)
    assert got[0] is None and got[1].data_ptr() == buf.data_ptr()
    # added before the rounding: one of the sum
    assert bool(((buf - (base + dw)).abs() <= U * (2 * base.abs() + 4 * dw.abs())).all())
    got = layers.linear_ce_backward(g, x, w, targets, lse, need_weight=False)
    assert got[1] is None and torch.equal(got[0], dx)
    one = layers.linear_ce_backward(torch.full((), 0.25, device="cuda").expand(500), x, w, targets, lse)
    many = layers.linear_ce_backward(torch.full((500,), 0.25, device="cuda"), x, w, targets, lse)
    assert all(torch.equal(a, b) for a, b in zip(one, many))


def test_gradients_of_small_and_large_scales():
    """fp16: losses weighted far below fp16's least number, and far above its largest, scaled out and in again."""
    x, w, targets, g = make(200, 900, 70, torch.float16, 2, pad=0.1)
    lse = layers.linear_ce_forward(x.cuda(), w.cuda(), targets.cuda())[1]
    a = layers.linear_ce_backward(g.cuda(), x.cuda(), w.cuda(), targets.cuda(), lse, grad_dtype=torch.float32)[1]
    for k in (-60, -20, 13, 40):
        b = layers.linear_ce_backward((g * 2.0 ** k).cuda(), x.cuda(), w.cuda(), targets.cuda(), lse, grad_dtype=torch.float32)[1]
        assert torch.equal(a * 2.0 ** k, b), k
    z = layers.linear_ce_backward((g * 0).cuda(), x.cuda(), w.cuda(), targets.cuda(), lse)
    assert not z[0].any() and not z[1].any()


def test_no_rows():
    x, w, targets = torch.empty(0, 50, device="cuda"), torch.ones(30, 50, device="cuda"), torch.empty(0, dtype=torch.int64, device="cuda")
    loss, lse = layers.linear_ce_forward(x, w, targets)
    assert loss.shape == lse.shape == (0,)
    dx, dw = layers.linear_ce_backward(loss, x, w, targets, lse)
    assert dx.shape == (0, 50) and dw.shape == (30, 50) and not dw.any()
    buf = torch.full((30, 50), 2.0, device="cuda")
    layers.linear_ce_backward(loss, x, w, targets, lse, grad_weight=buf, accumulate=True)
    assert bool((buf == 2.0).all())


def test_autograd_and_differences():
    """Gradients through autograd against central differences of the definition in 64 bits, in random directions."""
    x, w, targets, g = make(12, 90, 40, torch.float32, 21)
    gx, gw = x.view(3, 4, 40).cuda().requires_grad_(True), w.cuda().requires_grad_(True)
    loss = layers.linear_cross_entropy(gx, gw, targets.view(3, 4).cuda())
    assert loss.shape == (3, 4) and loss.dtype == torch.float32
    grads = torch.autograd.grad(loss, (gx, gw), g.view(3, 4).cuda())
    f = lambda x, w: (forward(x, w, targets)[0] * g.double()).sum()  # noqa: E731
    gen = torch.Generator().manual_seed(2)
    args = [x.double(), w.double()]
    for k, grad in enumerate(grads):
        d = torch.randn(args[k].shape, generator=gen, dtype=torch.float64)
        s = 1e-4
        want = (f(*[v if j != k else v + s * d for j, v in enumerate(args)]) - f(*[v if j != k else v - s * d for j, v in enumerate(args)])) / (2 * s)
        got = (grad.double().cpu().view(d.shape) * d).sum()
        # differences: s^2 of the third derivative (some times the value's size here), and 2^-52 / s; the gradient: its roundings
        assert abs(got - want) <= 1e-6 * (1 + abs(want)) + 200 * U * (grad.double().cpu().view(d.shape) * d).abs().sum(), (k, got, want)


def test_autograd_of_either_and_once():
    x, w, targets, g = (v.cuda() for v in make(50, 200, 64, torch.bfloat16, 12))
    _, lse = layers.linear_ce_forward(x, w, targets)
    want = layers.linear_ce_backward(g, x, w, targets, lse)
    for which in ((0,), (1,), (0, 1)):
        a = [v.detach().requires_grad_(k in which) for k, v in enumerate((x, w))]
        got = torch.autograd.grad(layers.linear_cross_entropy(*a, targets), [a[k] for k in which], g)
        assert all(torch.equal(v, want[k]) for v, k in zip(got, which))
    x.requires_grad_(True)
    grad, = torch.autograd.grad(layers.linear_cross_entropy(x, w, targets).sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="cannot be differentiated"):
        grad.float().sum().backward()
    loss = layers.linear_cross_entropy(x, w, targets)
    w.add_(1.0)
    with pytest.raises(RuntimeError, match="modified by an inplace"):
        loss.sum().backward()


def test_against_the_distillation_loss_of_one_target():
    """With logits in memory and a list of one entry, distill_loss is the same loss."""
    x, w, targets, _ = make(150, 800, 64, torch.float32, 17)
    z = (x.double() @ w.double().t()).float().cuda()
    a = layers.distill_loss(z, targets[:, None].cuda(), torch.zeros(150, 1).cuda())
    b = layers.linear_cross_entropy(x.cuda(), w.cuda(), targets.cuda())
    _, _, zz, ez, tl, *_ = forward(x, w, targets)
    assert bool(((a - b).abs().double().cpu() <= 2 * tl + 200 * U * (1 + a.double().cpu())).all())


def test_on_two_streams_and_in_a_graph():
    x, w, targets, g = (v.cuda() for v in make(700, 3000, 256, torch.bfloat16, 31))

    def run(x, targets):
        loss, lse = layers.linear_ce_forward(x, w, targets)
        return (loss, lse, *layers.linear_ce_backward(g, x, w, targets, lse))

    want, other = run(x, targets), run(x * 2, targets.flip(0))
    torch.cuda.synchronize()
    sides, keep = [torch.cuda.Stream(), torch.cuda.Stream()], []
    x2, t2 = x * 2, targets.flip(0)
    torch.cuda.synchronize()
    for _ in range(3):
        for side, args in zip(sides, ((x, targets), (x2, t2))):
            with torch.cuda.stream(side):
                keep.append(run(*args))
    torch.cuda.synchronize()
    for k, got in enumerate(keep):
        assert all(torch.equal(p, q) for p, q in zip(got, (want, other)[k % 2])), k
    xs, ts = x.clone(), targets.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run(xs, ts)
    for k in range(4):
        xs.copy_(x * (1 + 0.1 * k))
        ts.copy_(targets.roll(k))          # other rows to ignore at every replay
        eager = run(xs, ts)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(eager, out)), k


def test_weights_of_more_elements_than_32_bits_count():
    """2^31 + elements of weight and of its gradient (4.3 GB each in bf16): the last tiles against the same entries alone."""
    vocab, dim, n = (1 << 20) + 300, 2048, 40
    w = torch.zeros(vocab, dim, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(3)
    w[-300:] = torch.randn(300, dim, generator=g, device="cuda") * 0.2
    x = torch.randn(n, dim, generator=g, device="cuda").bfloat16()
    targets = torch.randint(vocab - 300, vocab, (n,), generator=g, device="cuda")
    loss, lse = layers.linear_ce_forward(x, w, targets)
    z = x.double() @ w[-300:].double().t()
    full = torch.logaddexp(torch.logsumexp(z, 1), torch.tensor(math.log(vocab - 300), device="cuda", dtype=torch.float64))
    want = full - z.gather(1, (targets - (vocab - 300))[:, None])[:, 0]
    e = 200 * U * (x.double().abs() @ w[-300:].double().abs().t()).max(1).values + 2000 * U * full
    assert bool(((loss.double() - want).abs() <= e).all())
    gl = torch.full((n,), 1.0 / n, device="cuda")
    dx, dw = layers.linear_ce_backward(gl, x, w, targets, lse)
    p = torch.exp(z - full[:, None])
    p.scatter_add_(1, (targets - (vocab - 300))[:, None], torch.full((n, 1), -1.0, device="cuda", dtype=torch.float64))
    ref = p.t() @ x.double() / n
    tol = 2.0 ** -8 * ref.abs() + (2.0 ** -8 + 2 * e.max()) * (p.abs().t() @ x.double().abs()) / n + 1e-30
    assert bool(((dw[-300:].double() - ref).abs() <= tol).all())


def test_refusals_of_the_tensors():
    x, w, t = torch.ones(4, 8, device="cuda"), torch.ones(5, 8, device="cuda"), torch.zeros(4, dtype=torch.int64, device="cuda")
    loss, lse = layers.linear_ce_forward(x, w, t)
    fwd, bwd = layers.linear_ce_forward, layers.linear_ce_backward
    for call in (lambda: fwd(x, w[:, :4], t), lambda: fwd(x, w.half(), t), lambda: fwd(x, w.cpu(), t), lambda: fwd(x, w, t[:2]), lambda: fwd(x, w, t.float()),
                 lambda: fwd(x.double(), w.double(), t), lambda: fwd(x, w[0], t), lambda: fwd(x, w[:0], t), lambda: fwd(x[0, 0], w, t),
                 lambda: bwd(loss[:2], x, w, t, lse), lambda: bwd(loss.double(), x, w, t, lse), lambda: bwd(loss, x, w, t, lse.cpu()),
                 lambda: bwd(loss, x, w, t, lse, accumulate=True), lambda: bwd(loss, x, w, t, lse, grad_weight=w[:4]),
                 lambda: bwd(loss, x, w, t, lse, grad_weight=w.double()), lambda: bwd(loss, x, w, t, lse, grad_dtype=torch.int32)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(L.LoptError, match="overlap"):
        bwd(loss, x, w, t, lse, grad_weight=w)


def test_probabilities_under_a_large_common_offset():
    """fp32 logits that are exact, 500 to 4000 above 0: with lse as it is kept, a probability is off by the roundings of a small
    difference, however large lse is.  dx under a weight's column of ones is what a token's gradients add up to."""
    from linear_ce_cases import product_depth
    n, vocab, dim = 200, 60, 48
    g = torch.Generator().manual_seed(16)
    x, w = torch.zeros(n, dim), torch.randint(-8, 9, (vocab, dim), generator=g) / 8.0
    x[:, 1:9] = torch.randint(-8, 9, (n, 8), generator=g) / 8.0
    x[:, 0], w[:, 0] = torch.randint(500 * 64, 4000 * 64, (n,), generator=g) / 64.0, 1.0
    targets, gl = torch.randint(0, vocab, (n,), generator=g), torch.rand(n, generator=g)
    z = x.double() @ w.double().t()
    assert torch.equal(z, z.float().double())
    lse = layers.linear_ce_forward(x.cuda(), w.cuda(), targets.cuda())[1]
    dx, dw = layers.linear_ce_backward(gl.cuda(), x.cuda(), w.cuda(), targets.cuda(), lse)
    d = z - lse.double().cpu()[:, None]
    p, gd = torch.exp(d.clamp(max=0.0)), gl.double()[:, None]
    G = gd * (p - torch.zeros_like(p).scatter_(1, targets[:, None], 1.0))
    # the difference, its product with log2(e) and that constant: U each of an exponent of |d|; the exponential 2 U, then two of G's own
    eG = gd * p * (3 * d.abs() + 4) * U + 2 * U * G.abs()
    close(dx, G @ w.double(), eG @ w.double().abs() + product_depth(vocab, torch.float32) * U * (G.abs() @ w.double().abs()), "dx")
    close(dw, G.t() @ x.double(), eG.t() @ x.double().abs() + product_depth(n, torch.float32) * U * (G.abs().t() @ x.double().abs()), "dw")
