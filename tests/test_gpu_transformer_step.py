"""A transformer's training step from the operators together: tokens -> embedding -> blocks joined by residual updates with
their norms -> cross entropy of the output layer -> gradients -> AdamW or the learned optimizer; eager through autograd, and
captured into one HIP graph."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - CPU container
    pytest.skip("no GPU", allow_module_level=True)

from adamw_cases import as_numpy, step_moments, step_param  # noqa: E402
from learned_optimizer_step_amd import layers  # noqa: E402
from learned_optimizer_step_amd import lopt as L  # noqa: E402
from learned_optimizer_step_amd import workloads as W  # noqa: E402
from ops_cases import U  # noqa: E402

VOCAB, DIM, TOKENS, BETA = 311, 96, 150, 0.7
NAMES = ("wte", "norm0", "w1", "post1", "gate1", "norm1", "w2", "post2", "norm2", "head")


def data(step):
    g = torch.Generator().manual_seed(100 + step)
    ids = torch.randint(-1, VOCAB, (TOKENS,), generator=g)
    targets = torch.randint(0, VOCAB, (TOKENS,), generator=g)
    targets[torch.rand(TOKENS, generator=g) < 0.2] = -1
    return ids, targets


def parameters():
    g = torch.Generator().manual_seed(1)
    vec = lambda m: m + 0.1 * torch.randn(DIM, generator=g)  # noqa: E731
    mat = lambda *s: torch.randn(*s, generator=g) * DIM ** -0.5  # noqa: E731
    return [torch.randn(VOCAB, DIM, generator=g) * 0.5, vec(1), mat(DIM, DIM), vec(1), vec(0.5), vec(1), mat(DIM, DIM), vec(1), vec(1), mat(VOCAB, DIM)]


def loss64(ps, ids, targets):
    """The run in 64 bits with torch's own operators."""
    wte, n0, w1, p1, g1, n1, w2, p2, n2, head = ps
    rms = lambda x, w: x * (x.square().mean(1, keepdim=True) + 1e-6).rsqrt() * w  # noqa: E731
    x = wte[ids.clamp(min=0)] * (ids >= 0)[:, None]
    z = rms(x, n0)
    x = x + BETA * g1 * rms(torch.tanh(z @ w1), p1)
    z = rms(x, n1)
    x = x + BETA * rms(torch.tanh(z @ w2), p2)
    z = rms(x, n2)
    return torch.nn.functional.cross_entropy(z @ head.t(), targets, ignore_index=-1, reduction="sum") / TOKENS


def run(ps, ids, targets):
    wte, n0, w1, p1, g1, n1, w2, p2, n2, head = ps
    x = layers.embedding(ids, wte)
    z = layers.rms_norm(x, n0, 1e-6)
    x, z = layers.residual_norm(x, torch.tanh(z @ w1), g1, p1, None, n1, None, 1e-6, beta=BETA, rms=True)
    _, z = layers.residual_norm(x, torch.tanh(z @ w2), None, p2, None, n2, None, 1e-6, beta=BETA, rms=True)
    return layers.linear_cross_entropy(z, head, targets).sum() / TOKENS


def test_gradients_of_the_run():
    ps = parameters()
    ids, targets = data(0)
    ps64 = [p.double().requires_grad_(True) for p in ps]
    want_loss = loss64(ps64, ids, targets)
    want = torch.autograd.grad(want_loss, ps64)
    gpu = [p.cuda().requires_grad_(True) for p in ps]
    loss = run(gpu, ids.cuda(), targets.cuda())
    got = torch.autograd.grad(loss, gpu)
    assert abs(loss.item() - want_loss.item()) <= 1e-5 * (1 + loss.item())
    for name, a, b in zip(NAMES, got, want):
        # two dozen operators of some hundred roundings each, on gradients whose entries are sums of both signs
        off = (a.double().cpu() - b).norm() / b.norm()
        assert off <= 4000 * U, (name, off.item())


@pytest.mark.parametrize("bits", [32, 8])
def test_steps_of_adamw(bits):
    """Training steps through autograd; every parameter after each against the definition on the same gradients."""
    ps = [p.cuda().requires_grad_(True) for p in parameters()]
    opt = L.AdamW(ps, lr=1e-2, weight_decay=0.1, state_bits=bits, seed=2)
    for t in (1, 2, 3):
        ids, targets = (v.cuda() for v in data(t))
        opt.zero_grad()
        run(ps, ids, targets).backward()
        before = [(as_numpy(p).reshape(-1).copy(), as_numpy(s).copy()) for p, s in zip(ps, opt.states)]
        opt.step()
        for k, (p, (old, state)) in enumerate(zip(ps, before)):
            n = p.numel()
            m, v, new = step_moments(as_numpy(p.grad).reshape(-1), state, bits, opt.betas, 2, t, k)
            assert (as_numpy(opt.states[k]) == new).all(), (t, NAMES[k])
            want, update = step_param(old, m.reshape(-1)[:n], v.reshape(-1)[:n], opt.betas, opt.eps, 1e-2, 0.1, t)
            assert (abs(as_numpy(p).reshape(-1) - want) <= U * (4 * abs(old) + 16 * update) + 1e-12).all(), (t, NAMES[k])


def test_the_learned_optimizer_steps_on_the_same_gradients():
    ps = [p.cuda().requires_grad_(True) for p in parameters()]
    opt = L.LearnedOptimizer(ps, W.mlp_weights(bias_std=0.1), lr=1.0)
    before = [p.detach().clone() for p in ps]
    ids, targets = (v.cuda() for v in data(1))
    run(ps, ids, targets).backward()
    opt.step()
    assert all(torch.isfinite(p).all() and not torch.equal(p, q) for p, q in zip(ps, before))
    opt.lopt.close()


@pytest.mark.parametrize("bits", [32, 8])
def test_a_whole_step_in_one_graph(bits):
    """Forward, backward and AdamW's step captured once; every replay against the same calls made eagerly on another copy,
    bit for bit.  Other rows are ignored in every step."""

    class Side:
        def __init__(self):
            self.p = [v.cuda() for v in parameters()]
            self.g = [torch.zeros_like(v) for v in self.p]
            self.s = [layers.adamw_state(v, bits) for v in self.p]
            self.step_count = torch.zeros(2, dtype=torch.int64, device="cuda")
            self.ids, self.targets = (v.cuda() for v in data(0))
            self.dl = torch.full((TOKENS,), 1.0 / TOKENS, device="cuda")
            self.loss = None

        def step(self):
            wte, n0, w1, p1, g1, n1, w2, p2, n2, head = self.p
            o = dict(beta=BETA, rms=True)
            x0 = layers.embedding_forward(self.ids, wte)
            z0, _, r0 = layers.norm_forward(x0, n0, None, 1e-6, rms=True)
            y1 = torch.tanh(z0 @ w1)
            x1, z1, s1 = layers.residual_norm_forward(x0, y1, g1, p1, None, n1, None, 1e-6, **o)
            y2 = torch.tanh(z1 @ w2)
            x2, z2, s2 = layers.residual_norm_forward(x1, y2, None, p2, None, n2, None, 1e-6, **o)
            self.loss, lse = layers.linear_ce_forward(z2, head, self.targets)
            dz2, _ = layers.linear_ce_backward(self.dl, z2, head, self.targets, lse, grad_weight=self.g[9])
            dx1, dy2, *_ = layers.residual_norm_backward(None, dz2, y2, x2, s2, None, p2, None, n2, grad_post_weight=self.g[7],
                                                         grad_weight=self.g[8], **o)
            dy2 = dy2 * (1 - y2 * y2)
            torch.mm(z1.t().contiguous(), dy2, out=self.g[6])
            dz1 = dy2 @ w2.t().contiguous()
            dx0, dy1, *_ = layers.residual_norm_backward(dx1, dz1, y1, x1, s1, g1, p1, None, n1, grad_gate=self.g[4],
                                                         grad_post_weight=self.g[3], grad_weight=self.g[5], **o)
            dy1 = dy1 * (1 - y1 * y1)
            torch.mm(z0.t().contiguous(), dy1, out=self.g[2])
            dn, _, _ = layers.norm_backward(dy1 @ w1.t().contiguous(), x0, n0, None, r0, rms=True, grad_weight=self.g[1])
            layers.embedding_backward(dx0 + dn, self.ids, VOCAB, out=self.g[0])
            layers.adamw_step(self.p, self.g, self.s, self.step_count, lr=1e-2, weight_decay=0.1, state_bits=bits, seed=5)

        def feed(self, t):
            for to, v in zip((self.ids, self.targets), data(t)):
                to.copy_(v)

    eager, graphed = Side(), Side()
    for s in (eager, graphed):
        s.step()          # the libraries' own first calls
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        graphed.step()
    for t in range(1, 6):
        eager.feed(t)
        graphed.feed(t)
        eager.step()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(eager.loss, graphed.loss), t
        for a, b in zip(eager.g + eager.p + eager.s, graphed.g + graphed.p + graphed.s):
            assert torch.equal(a, b), t
    assert eager.step_count.tolist() == graphed.step_count.tolist() == [6, 0]


def test_gradients_into_the_same_buffers_of_two_batches():
    """Two batches' gradients added up in one set of buffers, as one call of both batches gives them."""
    ids, targets = (v.cuda() for v in data(3))
    g = torch.Generator().manual_seed(7)
    z, head = torch.randn(TOKENS, DIM, generator=g).cuda(), parameters()[9].cuda()
    loss, lse = layers.linear_ce_forward(z, head, targets)
    dl = torch.full((TOKENS,), 1.0 / TOKENS, device="cuda")
    _, want = layers.linear_ce_backward(dl, z, head, targets, lse)
    buf = torch.zeros_like(head)
    for part in (slice(0, 70), slice(70, TOKENS)):
        layers.linear_ce_backward(dl[part], z[part], head, targets[part], lse[part], grad_weight=buf, accumulate=True)
    # sums of the same terms in another order
    assert bool(((buf - want).abs() <= 400 * U * (want.abs() + want.abs().max())).all())


def test_steps_of_adamw_with_8_bit_moments():
    """Training steps through autograd: codes of the fp32 moments and their random bits, and the parameters they move."""
    from test_gpu_adamw import fp32_codes
    ps = [p.cuda().requires_grad_(True) for p in parameters()]
    opt = L.AdamW(ps, lr=1e-2, weight_decay=0.1, state_bits=8, seed=2)
    for t in (1, 2, 3):
        ids, targets = (v.cuda() for v in data(t))
        opt.zero_grad()
        run(ps, ids, targets).backward()
        before = [(as_numpy(p).reshape(-1).copy(), as_numpy(s).copy()) for p, s in zip(ps, opt.states)]
        opt.step()
        for k, (p, (old, state)) in enumerate(zip(ps, before)):
            m, v, new = fp32_codes(as_numpy(p.grad).reshape(-1), state, 2, t, k)
            assert (as_numpy(opt.states[k]) == new).all(), (t, NAMES[k])
            want, update = step_param(old, m.reshape(-1)[:p.numel()], v.reshape(-1)[:p.numel()], opt.betas, opt.eps, 1e-2, 0.1, t)
            assert (abs(as_numpy(p).reshape(-1) - want) <= U * (4 * abs(old) + 16 * update) + 1e-12).all(), (t, NAMES[k])
