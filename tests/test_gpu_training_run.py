"""The operators together, as a training step uses them: tokens -> embedding ->
norms -> logits -> distillation loss -> gradients -> the learned optimizer's
step; eager through autograd, and captured into one HIP graph with gradients
kept in the buffers that the step reads."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - CPU container
    pytest.skip("no GPU", allow_module_level=True)

import oracle  # noqa: E402
from learned_optimizer_step_amd import layers  # noqa: E402
from learned_optimizer_step_amd import lopt as L  # noqa: E402
from learned_optimizer_step_amd import workloads as W  # noqa: E402
from ops_cases import U, distill  # noqa: E402

VOCAB, DIM, TOKENS, TOP, TAU = 211, 96, 150, 9, 2.0
SCALE = DIM ** 0.5


def data(step):
    g = torch.Generator().manual_seed(100 + step)
    ids = torch.randint(-1, VOCAB, (TOKENS,), generator=g)
    tid = torch.rand(TOKENS, VOCAB, generator=g).argsort(1)[:, :TOP]
    tid[torch.rand(TOKENS, TOP, generator=g) < 0.2] = -1
    return ids, tid, torch.randn(TOKENS, TOP, generator=g) * 2


def parameters():
    g = torch.Generator().manual_seed(1)
    emb = torch.randn(VOCAB, DIM, generator=g) * 0.05
    return [emb, 1 + 0.1 * torch.randn(DIM, generator=g), 0.1 * torch.randn(DIM, generator=g),
            1 + 0.1 * torch.randn(DIM, generator=g), torch.randn(DIM, VOCAB, generator=g) * 0.1]


def loss64(ps, ids, tid, tu):
    """The run in 64 bits with torch's own operators."""
    emb, lw, lb, rw, head = ps
    x = emb[ids.clamp(min=0)] * SCALE * (ids >= 0)[:, None]
    x = torch.nn.functional.layer_norm(x, (DIM,), lw, lb, 1e-5)
    x = x * (x.square().mean(1, keepdim=True) + 1e-6).rsqrt() * rw
    z = x @ head
    there = tid >= 0
    p = torch.where(there.any(1, keepdim=True), torch.where(there, tu.double() / TAU, -float("inf")), 0.0).softmax(1) * there
    logq = torch.log_softmax(z / TAU, 1).gather(1, tid.clamp(min=0))
    return (TAU * TAU * (torch.special.xlogy(p, p) - p * logq).sum(1)).mean()


def run(ps, ids, tid, tu):
    emb, lw, lb, rw, head = ps
    x = layers.embedding(ids, emb, SCALE)
    x = layers.rms_norm(layers.layer_norm(x, lw, lb, 1e-5), rw, 1e-6)
    return layers.distill_loss(x @ head, tid, tu, TAU).mean()


def test_gradients_of_the_run():
    ps = parameters()
    ids, tid, tu = data(0)
    ps64 = [p.double().requires_grad_(True) for p in ps]
    want = torch.autograd.grad(loss64(ps64, ids, tid, tu), ps64)
    gpu = [p.cuda().requires_grad_(True) for p in ps]
    loss = run(gpu, ids.cuda(), tid.cuda(), tu.cuda())
    got = torch.autograd.grad(loss, gpu)
    assert abs(loss.item() - loss64(ps64, ids, tid, tu).item()) <= 1e-5 * (1 + loss.item())
    for k, (a, b) in enumerate(zip(got, want)):
        # a dozen operators of some hundred roundings each, on gradients whose entries are sums of both signs
        off = (a.double().cpu() - b).norm() / b.norm()
        assert off <= 2000 * U, (k, off.item())


def test_steps_of_the_learned_optimizer():
    """Three training steps: the parameters after each against the oracle's step on the same gradients, and a loss that
    autograd can go through every time."""
    mlp = W.mlp_weights(bias_std=0.1)
    ps = [p.cuda().requires_grad_(True) for p in parameters()]
    opt = L.LearnedOptimizer(ps, mlp, lr=1.0)
    host = [p.detach().cpu().numpy().copy() for p in ps]
    shape = [L.matrix_shape(p.shape) for p in ps]
    host = [h.reshape(s) for h, s in zip(host, shape)]
    states = [{"m": np.zeros((3, *s), np.float32), "v": np.zeros(s, np.float32), "r": np.zeros((3, s[0]), np.float32),
               "c": np.zeros((3, s[1]), np.float32)} for s in shape]
    for t in (1, 2, 3):
        ids, tid, tu = (v.cuda() for v in data(t))
        opt.zero_grad()
        run(ps, ids, tid, tu).backward()
        grads = [p.grad.cpu().numpy().reshape(s) for p, s in zip(ps, shape)]
        assert all(np.isfinite(g).all() and np.abs(g).max() > 0 for g in grads)
        opt.step()
        host, states = oracle.step(host, grads, states, t, mlp, oracle.Hyper())
        for p, h in zip(ps, host):
            got = p.detach().cpu().numpy().reshape(h.shape).astype(np.float64)
            assert np.all(np.abs(got - h) <= 1e-7 + 1e-5 * np.abs(h))
    opt.lopt.close()


def test_a_whole_step_in_one_graph():
    """Forward, backward and the optimizer's step captured once; every replay against the same calls made eagerly on
    another copy of the parameters, bit for bit."""
    mlp = W.mlp_weights(bias_std=0.1)

    class Side:
        def __init__(self):
            self.p = [v.cuda() for v in parameters()]
            self.g = [torch.zeros_like(v) for v in self.p]
            self.opt = L.LOpt(self.p, mlp)
            self.ids, self.tid, self.tu = (v.cuda() for v in data(0))
            self.dl = torch.full((TOKENS,), 1.0 / TOKENS, device="cuda")
            self.loss = None

        def step(self):
            emb, lw, lb, rw, head = self.p
            x0 = layers.embedding_forward(self.ids, emb, SCALE)
            x1, mean, rstd = layers.norm_forward(x0, lw, lb, 1e-5)
            x2, _, rstd2 = layers.norm_forward(x1, rw, None, 1e-6, rms=True)
            z = x2 @ head
            self.loss, lse = layers.distill_forward(z, self.tid, self.tu, TAU)
            dz = layers.distill_backward(self.dl, z, self.tid, self.tu, lse, TAU, out=z)
            torch.mm(x2.t().contiguous(), dz, out=self.g[4])
            dx2 = dz @ head.t().contiguous()
            dx1, _, _ = layers.norm_backward(dx2, x1, rw, None, rstd2, rms=True, grad_weight=self.g[3])
            dx0, _, _ = layers.norm_backward(dx1, x0, lw, mean, rstd, grad_weight=self.g[1], grad_bias=self.g[2])
            layers.embedding_backward(dx0, self.ids, VOCAB, SCALE, out=self.g[0])
            self.opt.step(self.g)

        def feed(self, t):
            for to, v in zip((self.ids, self.tid, self.tu), data(t)):
                to.copy_(v)

    eager, graphed = Side(), Side()
    for s in (eager, graphed):
        s.feed(0)
        s.step()          # binds the gradients' addresses before the capture
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
        for k in range(5):
            assert torch.equal(eager.g[k], graphed.g[k]), (t, k)
            assert torch.equal(eager.p[k], graphed.p[k]), (t, k)
    assert eager.opt.t == graphed.opt.t == 6
    eager.opt.close()
    graphed.opt.close()


def test_two_streams_at_once():
    """The same operators on two streams that overlap, each with its own data: as one after the other."""
    keep = []   # the inputs belong to the default stream: they must outlive the other's work

    def work(seed, stream=None):
        g = torch.Generator(device="cuda").manual_seed(seed)
        n, vocab, dim = 9000 + seed, 3000, 256
        ids = torch.randint(-1, vocab, (n,), generator=g, device="cuda")
        x = torch.randn(n, dim, generator=g, device="cuda").bfloat16()
        w = torch.randn(dim, generator=g, device="cuda")
        z = torch.randn(700, 5000, generator=g, device="cuda").bfloat16()
        tid = torch.randint(-1, 5000, (700, 40), generator=g, device="cuda")
        tu = torch.randn(700, 40, generator=g, device="cuda")
        keep.append((ids, x, w, z, tid, tu))
        torch.cuda.current_stream().synchronize()   # the inputs are there; the other stream may still run
        with torch.cuda.stream(stream):
            for _ in range(4):
                y, mean, rstd = layers.norm_forward(x, w, w)
                dx, dw, db = layers.norm_backward(x, x, w, mean, rstd)
                dt = layers.embedding_backward(dx, ids, vocab, 2.0)
                loss, lse = layers.distill_forward(z, tid, tu, 2.0)
                dz = layers.distill_backward(loss, z, tid, tu, lse, 2.0)
        return y, dx, dw, db, dt, loss, lse, dz

    want = [work(1), work(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [work(1, streams[0]), work(2, streams[1])]
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert [torch.equal(p, q) for p, q in zip(a, b)] == [True] * 8


def test_distill_definition_of_the_tests():
    """The 64-bit definition that the distillation tests use, against torch's own operators."""
    ids, tid, tu = data(3)
    z = torch.randn(TOKENS, VOCAB, dtype=torch.float64, generator=torch.Generator().manual_seed(4)).requires_grad_(True)
    there = tid >= 0
    p = torch.where(there.any(1, keepdim=True), torch.where(there, tu.double() / TAU, -float("inf")), 0.0).softmax(1) * there
    logq = torch.log_softmax(z / TAU, 1).gather(1, tid.clamp(min=0))
    loss = TAU * TAU * (torch.special.xlogy(p, p) - p * logq).sum(1)
    grad, = torch.autograd.grad(loss.sum(), z)
    got = distill(z.detach(), tid, tu, TAU)
    assert torch.allclose(got[0], loss, rtol=1e-12, atol=1e-12) and torch.allclose(got[2] * TAU, grad, rtol=1e-10, atol=1e-13)


def test_gradients_through_autograd_in_a_graph():
    """Forward and backward through autograd captured once, replayed on new tokens; each replay against the same run made
    eagerly on copies of the parameters."""
    ps = [p.cuda().requires_grad_(True) for p in parameters()]
    copies = [p.detach().clone().requires_grad_(True) for p in ps]
    ids, tid, tu = (v.cuda() for v in data(0))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):      # the products' library is loaded before the capture
        torch.autograd.grad(run(copies, ids, tid, tu), copies)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        loss = run(ps, ids, tid, tu)
        grads = torch.autograd.grad(loss, ps)
        loss = loss.detach()
    for t in range(1, 5):
        for to, v in zip((ids, tid, tu), data(t)):
            to.copy_(v)
        want_loss = run(copies, ids, tid, tu)
        want = torch.autograd.grad(want_loss, copies)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(loss, want_loss.detach()), t
        assert [torch.equal(a, b) for a, b in zip(grads, want)] == [True] * 5, t
