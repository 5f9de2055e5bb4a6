"""AdamW on the GPU: moments and codes to the last bit, parameters against the definition in 64 bits."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - CPU container
    pytest.skip("no GPU", allow_module_level=True)

from adamw_cases import BLOCK, as_numpy, decode, decode_codes, encode, random_bits, step_moments, step_param  # noqa: E402
from learned_optimizer_step_amd import layers  # noqa: E402
from learned_optimizer_step_amd import lopt as L  # noqa: E402
from ops_cases import TINY, TYPES, U, half  # noqa: E402

BETAS, EPS = (0.9, 0.999), 1e-8
# one element, blocks and chunks with their neighbours, and lengths that no vector divides
SIZES = [1, 3, 255, 256, 257, 1023, 1024, 1025, 5000, 100_003]


def close_param(got, want, update, p, t, what):
    """A dozen fp32 roundings of the update, three of p, and the last one's to p's type."""
    tol = half(t) * np.abs(want) + TINY[t] + U * (3 * np.abs(p) + 16 * update)
    off = np.abs(as_numpy(got).astype(np.float64) - want)
    assert (off <= tol).all(), f"{what}: {np.max(off / tol):.3g} times the bound"


def make(sizes, pt, gt, bits, seed, warm=True):
    g = torch.Generator().manual_seed(seed)
    ps = [(0.1 * torch.randn(n, generator=g)).to(pt).cuda() for n in sizes]
    gs = [(torch.randn(n, generator=g) * 10.0 ** torch.randint(-4, 1, (n,), generator=g)).to(gt).cuda() for n in sizes]
    return ps, gs, [layers.adamw_state(p, bits) for p in ps]


def step_and_check(ps, gs, states, step, bits, lr, wd, seed, what):
    n = len(ps)
    lrs, wds = (np.broadcast_to(np.asarray(v, np.float64), n) for v in (lr, wd))
    before = [as_numpy(p).copy() for p in ps], [as_numpy(s).copy() for s in states]
    layers.adamw_step(ps, gs, states, step, lr=lr, betas=BETAS, eps=EPS, weight_decay=wd, state_bits=bits, seed=seed)
    t = int(step[0])
    assert int(step[1]) == 0
    for k in range(n):
        if gs[k] is None:
            assert np.array_equal(as_numpy(ps[k]), before[0][k]) and np.array_equal(as_numpy(states[k]), before[1][k])
            continue
        m, v, new = step_moments(as_numpy(gs[k]).reshape(-1), before[1][k], bits, BETAS, seed, t, k)
        assert np.array_equal(as_numpy(states[k]), new), f"{what} tensor {k}: moments differ"
        size = ps[k].numel()
        want, update = step_param(before[0][k].reshape(-1), m.reshape(-1)[:size], v.reshape(-1)[:size], BETAS, EPS, lrs[k], wds[k], t)
        close_param(ps[k].reshape(-1), want, update, before[0][k].reshape(-1), ps[k].dtype, f"{what} tensor {k}")


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("gt", TYPES, ids=str)
@pytest.mark.parametrize("pt", TYPES, ids=str)
def test_against_the_definition(pt, gt, bits):
    ps, gs, states = make(SIZES, pt, gt, bits, 3)
    step = torch.zeros(2, dtype=torch.int64, device="cuda")
    for t in range(3):
        step_and_check(ps, gs, states, step, bits, 1e-2, 0.1, 77, f"step {t}")
        gs = [g.flip(0) * 0.5 for g in gs]
    assert int(step[0]) == 3


def test_codes_that_fp32_rounds_up_to():
    """So many elements that some v in fp32 lie on a code's border while the definition's are below it."""
    n = 1 << 23
    ps, gs, states = make([n], torch.float32, torch.float32, 8, 21)
    step = torch.zeros(2, dtype=torch.int64, device="cuda")
    layers.adamw_step(ps, gs, states, step, lr=1e-3, betas=BETAS, eps=EPS, weight_decay=0.0, state_bits=8, seed=5)
    gs = [g.flip(0) for g in gs]
    v = decode(as_numpy(states[0]), 8)[1]
    step_and_check(ps, gs, states, step, 8, 1e-3, 0.0, 5, "borders")
    g = as_numpy(gs[0]).reshape(-1, BLOCK)
    u = (random_bits(5, 2, 0, 0, n).reshape(-1, BLOCK) >> np.uint64(16)).astype(np.float64) / 65536
    codes = []
    for x in (BETAS[1] * v + (1 - BETAS[1]) * g.astype(np.float64) ** 2,
              (v.astype(np.float32) * np.float32(BETAS[1]) + g * g * np.float32(1 - BETAS[1])).astype(np.float64)):
        code, e = encode(x, 31, u)
        codes.append(decode_codes(np.where((x > 0) & (code == 0), 1, code), e, 31))   # a v that is not 0 has a code that is not
    got = decode(as_numpy(states[0]), 8)[1]
    assert (got != codes[1]).any() and (got != codes[0]).sum() < (codes[1] != codes[0]).sum()


@pytest.mark.parametrize("bits", [32, 8])
def test_long_lists_of_several_types_and_skipped_tensors(bits):
    """More tensors than one launch takes, four pairs of types, rates of their own, none for some gradients."""
    g = torch.Generator().manual_seed(9)
    sizes = torch.randint(1, 3000, (391,), generator=g).tolist()
    ps, gs, states = [], [], []
    for k, n in enumerate(sizes):
        p, d, s = make([n], TYPES[k % 3], TYPES[0 if k % 2 else k % 3], bits, k)
        ps, gs, states = ps + p, gs + ([None] if k % 7 == 3 else d), states + s
    lr, wd = (1e-2 * torch.rand(391, generator=g)).tolist(), (0.2 * torch.rand(391, generator=g)).tolist()
    step = torch.zeros(2, dtype=torch.int64, device="cuda")
    for t in range(2):
        step_and_check(ps, gs, states, step, bits, lr, wd, 5, f"step {t}")


def test_all_skipped_and_empty_lists():
    ps, gs, states = make([300, 5], torch.float32, torch.float32, 32, 0)
    step = torch.zeros(2, dtype=torch.int64, device="cuda")
    layers.adamw_step(ps, [None, None], states, step, lr=1.0)
    assert step.tolist() == [1, 0]
    layers.adamw_step([], [], [], step, lr=1.0)
    assert step.tolist() == [1, 0]


@pytest.mark.parametrize("bits", [32, 8])
def test_unaligned_tensors_and_what_lies_around_them(bits):
    """Parameters and gradients at every element of a 16-byte piece; the elements before and behind stay as they were."""
    for t in TYPES:
        for off in range(1, 9):
            n = 1500 + off
            base = torch.full((n + 32,), 3.0, dtype=t, device="cuda")
            p = base[off:off + n]
            p.copy_(torch.randn(n))
            wide = torch.full((n + 32,), 7.0, dtype=t, device="cuda")
            g = wide[8 - off:8 - off + n]
            g.copy_(torch.randn(n))
            around = torch.full((40 * 528,), 9, dtype=torch.uint8, device="cuda")
            if bits == 8:
                state = around[16:16 + L.lopt_adamw_state_bytes(n, 8)]
                state.zero_()
            else:
                state = layers.adamw_state(p, bits)
            step = torch.zeros(2, dtype=torch.int64, device="cuda")
            step_and_check([p], [g], [state], step, bits, 1e-2, 0.0, 1, f"{t} at {off}")
            p.fill_(3.0)
            assert bool((base == 3.0).all())
            if bits == 8:
                state.fill_(9)
                assert bool((around == 9).all())


def test_gradients_of_any_layout():
    p = torch.randn(40, 30, device="cuda")
    g = torch.randn(30, 40, device="cuda").t()
    state = layers.adamw_state(p)
    step = torch.zeros(2, dtype=torch.int64, device="cuda")
    step_and_check([p], [g], [state], step, 32, 1e-2, 0.0, 0, "transposed")
    step_and_check([p], [torch.ones((), device="cuda").expand(40, 30)], [state], step, 32, 1e-2, 0.0, 0, "expanded")


def test_sizes_of_moments():
    """Gradients from the least to the largest floats, zeros among them: exponents at both ends of their range."""
    g = torch.Generator().manual_seed(31)
    x = torch.randn(64 * BLOCK, generator=g) * 2.0 ** torch.randint(-60, 60, (64, 1), generator=g).float().expand(64, BLOCK).reshape(-1)
    x[torch.rand(64 * BLOCK, generator=g) < 0.1] = 0.0
    x[:BLOCK] = 0.0
    x[BLOCK:2 * BLOCK] = 1.5e19           # v up to 2^127
    x[2 * BLOCK:3 * BLOCK] = 3e38 * torch.rand(BLOCK, generator=g)   # m up to 2^124, v infinite
    x[3 * BLOCK:4 * BLOCK] = 1e-18 * torch.rand(BLOCK, generator=g)
    x[4 * BLOCK] = 1.0                     # one large number among small ones
    x[4 * BLOCK + 1:5 * BLOCK] = 1e-6
    for bits in (32, 8):
        p = torch.zeros(64 * BLOCK, device="cuda")
        state, step = layers.adamw_state(p, bits), torch.zeros(2, dtype=torch.int64, device="cuda")
        for t in range(2):
            before = as_numpy(state).copy()
            layers.adamw_step([p], [x.cuda()], [state], step, lr=0.0, state_bits=bits, seed=4, weight_decay=0.0)
            _, _, new = step_moments(x.numpy(), before, bits, BETAS, 4, t + 1, 0)
            assert np.array_equal(as_numpy(state), new, equal_nan=bits == 32), (bits, t)
        m, v = layers.adamw_moments(state, p.numel(), state_bits=bits)
        wm, wv = decode(as_numpy(state), bits)
        assert np.array_equal(m.cpu().numpy(), wm.reshape(-1).astype(np.float32), equal_nan=True)
        assert np.array_equal(v.cpu().numpy(), wv.reshape(-1).astype(np.float32), equal_nan=True)


def test_moments_in_other_types():
    ps, gs, states = make([1000], torch.float32, torch.float32, 8, 8)
    layers.adamw_step(ps, gs, states, torch.zeros(2, dtype=torch.int64, device="cuda"), lr=0.1, state_bits=8)
    m, v = layers.adamw_moments(states[0], 1000, state_bits=8)
    for t in (torch.bfloat16, torch.float16):
        a, b = layers.adamw_moments(states[0], 1000, state_bits=8, dtype=t)
        assert torch.equal(a, m.to(t)) and torch.equal(b, v.to(t))
    a, b = layers.adamw_moments(states[0], 1000, state_bits=8, dtype=torch.bfloat16)
    assert torch.equal(a.float(), m) and torch.equal(b.float(), v)


def test_nan_and_infinity_stay_in_their_place():
    """32-bit moments: the element's own; 8-bit ones: its block's of 256."""
    for bad in (float("nan"), float("inf"), -float("inf")):
        for bits in (32, 8):
            ps, gs, states = make([2000], torch.float32, torch.float32, bits, 2)
            gs[0][700] = bad
            step = torch.zeros(2, dtype=torch.int64, device="cuda")
            for _ in range(2):
                layers.adamw_step(ps, gs, states, step, lr=1e-3, state_bits=bits)
                gs[0][700] = 0.25
            lost = ~torch.isfinite(layers.adamw_moments(states[0], 2000, state_bits=bits)[0])
            want = torch.zeros(2000, dtype=torch.bool)
            want[slice(512, 768) if bits == 8 else 700] = True
            assert torch.equal(lost.cpu(), want), (bad, bits)
            assert torch.equal(~torch.isfinite(ps[0]).cpu() | want, want)


def test_codes_keep_the_mean():
    """A number between two codes becomes either with the probability that keeps its mean: over 2^20 elements of one value
    the mean is off by at most 6 deviations of a step's half, and by the 2^-16 of a step that 16 bits leave out."""
    n = 1 << 20
    for x in (0.7321, 0.031, 1e-3):
        g = torch.full((n,), x, device="cuda")
        g[::BLOCK] = 1.0                   # the block's exponent
        p = torch.zeros(n, device="cuda")
        state = layers.adamw_state(p, 8)
        layers.adamw_step([p], [g], [state], torch.zeros(2, dtype=torch.int64, device="cuda"), lr=0.0, state_bits=8, seed=11)
        keep = torch.ones(n, dtype=torch.bool, device="cuda")
        keep[::BLOCK] = False
        for got, want in zip(layers.adamw_moments(state, n, state_bits=8), (0.1 * x, 0.001 * x * x)):
            got = got[keep].double()
            assert 2 == len(got.unique()) and got.min() <= want <= got.max()
            gap = (got.max() - got.min()).item()
            assert abs(got.mean().item() - want) <= gap * (6 * 0.5 / n ** 0.5 + 2.0 ** -16) + 1e-7 * want


def test_second_moments_decay():
    """Without gradients v falls by 0.999 a step on average, though a code's step is a tenth: 500 steps from one value. The
    codes' random walk: each step adds at most 0.001 v of a step of v / 8 or less, a variance of 0.000125 v^2 an element."""
    n = 1 << 16
    p, g = torch.zeros(n, device="cuda"), torch.ones(n, device="cuda")
    state, step = layers.adamw_state(p, 8), torch.zeros(2, dtype=torch.int64, device="cuda")
    layers.adamw_step([p], [g], [state], step, lr=0.0, state_bits=8)
    v0 = layers.adamw_moments(state, n, state_bits=8)[1].double().mean().item()
    g.zero_()
    for _ in range(500):
        layers.adamw_step([p], [g], [state], step, lr=0.0, state_bits=8)
    v = layers.adamw_moments(state, n, state_bits=8)[1].double().mean().item()
    want = v0 * 0.999 ** 500
    assert abs(v / want - 1) <= 6 * (500 * 0.000125 / n) ** 0.5 * v0 / want + 500 * 2.0 ** -16 / 8


def test_more_elements_than_32_bits_count():
    """2^32 + 700 elements: the first and the last blocks against the definition."""
    n = (1 << 32) + 700
    p = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    g = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    part = torch.randn(2 * BLOCK, device="cuda").bfloat16()
    for at in (0, n - 700):
        g[at:at + 2 * BLOCK] = part
    state, step = layers.adamw_state(p, 8), torch.zeros(2, dtype=torch.int64, device="cuda")
    layers.adamw_step([p], [g], [state], step, lr=1e-2, state_bits=8, seed=3, weight_decay=0.0)
    rows = state.view(-1, 528)
    for at in (0, n - 700):
        m, v, new = step_moments(as_numpy(part), np.zeros(2 * 528, np.uint8), 8, BETAS, 3, 1, 0, at)
        got = rows[at // BLOCK:at // BLOCK + 2].cpu().numpy().reshape(-1)
        assert np.array_equal(got, new)
        want, update = step_param(np.zeros(2 * BLOCK), m.reshape(-1), v.reshape(-1), BETAS, EPS, 1e-2, 0.0, 1)
        close_param(p[at:at + 2 * BLOCK], want, update, np.zeros(2 * BLOCK), torch.bfloat16, f"at {at}")
    assert not p[2 * BLOCK:n - 700].any()


@pytest.mark.parametrize("bits", [32, 8])
def test_in_a_graph(bits):
    """A captured step counts on: replays against eager steps on a copy, gradients and a schedule's rate changing between."""
    sizes = [700] * 100 + [5000, 3]
    sides = [make(sizes, torch.float32, torch.float32, bits, 6) for _ in range(2)]
    steps = [torch.zeros(2, dtype=torch.int64, device="cuda") for _ in range(2)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layers.adamw_step(*sides[1], steps[1], lr=1e-2, state_bits=bits, seed=8)
    assert int(steps[1][0]) == 0
    for k in range(5):
        for ps, gs, _ in sides:
            for i, g in enumerate(gs):
                g.mul_(0.5).add_(0.01 * (i % 5) * (k + 1))
        layers.adamw_step(*sides[0], steps[0], lr=1e-2, state_bits=bits, seed=8)
        graph.replay()
        torch.cuda.synchronize()
        assert steps[0].tolist() == steps[1].tolist() == [k + 1, 0]
        for a, b in zip(sides[0][0] + sides[0][2], sides[1][0] + sides[1][2]):
            assert torch.equal(a, b), k


def test_two_streams_at_once():
    sides = [make([3_000_000, 70, 256], torch.float32, torch.float32, 8, 20 + k) for k in range(2)]
    want = []
    for ps, gs, states in sides:
        ps, states = [p.clone() for p in ps], [s.clone() for s in states]
        step = torch.zeros(2, dtype=torch.int64, device="cuda")
        for _ in range(4):
            layers.adamw_step(ps, gs, states, step, lr=1e-2, state_bits=8)
        want.append(ps + states)
    torch.cuda.synchronize()
    steps = [torch.zeros(2, dtype=torch.int64, device="cuda") for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(4):
        for side, step, stream in zip(sides, steps, streams()):
            with torch.cuda.stream(stream):
                layers.adamw_step(*side, step, lr=1e-2, state_bits=8)
    torch.cuda.synchronize()
    for side, w in zip(sides, want):
        assert all(torch.equal(a, b) for a, b in zip(side[0] + side[2], w))


def streams(made=[]):
    made += [torch.cuda.Stream() for _ in range(2 - len(made))]
    return made


def test_extreme_settings():
    """beta 0 (no average and no correction), lr 0 (moments only), far steps."""
    ps, gs, states = make([900], torch.float32, torch.float32, 32, 12)
    p0, step = ps[0].clone(), torch.zeros(2, dtype=torch.int64, device="cuda")
    layers.adamw_step(ps, gs, states, step, lr=1e-2, betas=(0.0, 0.0), eps=0.0, weight_decay=0.0)
    want = p0.double() - 1e-2 * torch.sign(gs[0]).double()
    assert bool(((ps[0].double() - want).abs() <= U * (3 * p0.double().abs() + 0.16)).all())
    before = ps[0].clone()
    layers.adamw_step(ps, gs, states, step, lr=0.0, weight_decay=0.3)
    assert torch.equal(ps[0], before)
    step[0] = 1 << 40
    layers.adamw_step(ps, gs, states, step, lr=1e-2)
    assert torch.isfinite(ps[0]).all() and int(step[0]) == (1 << 40) + 1


# ---- lopt.AdamW

def test_the_optimizer_and_its_schedule():
    """Groups with their own decay, a schedule of rates, a parameter without a gradient, against the definition."""
    g = torch.Generator().manual_seed(2)
    w, b, idle = (torch.randn(s, generator=g).cuda().requires_grad_(True) for s in ((33, 20), (20,), (7,)))
    opt = L.AdamW([{"params": [w], "weight_decay": 0.1}, {"params": [b, idle], "weight_decay": 0.0}], lr=0.1, state_bits=8, seed=6)
    sched = torch.optim.lr_scheduler.CosineAnnealingLR(opt, T_max=5)
    for t in range(1, 4):
        lr = opt.param_groups[0]["lr"]
        opt.zero_grad()
        (w.square().sum() + (b * 3).sum()).backward()
        before = [as_numpy(x).copy() for x in (w, b, *opt.states)]
        grads = [as_numpy(x.grad).reshape(-1) for x in (w, b)]
        opt.step()
        sched.step()
        for k, (x, wd) in enumerate(((w, 0.1), (b, 0.0))):
            n = x.numel()
            m, v, new = step_moments(grads[k], before[2 + k], 8, BETAS, 6, t, k)
            assert np.array_equal(as_numpy(opt.states[k]), new)
            want, update = step_param(before[k].reshape(-1), m.reshape(-1)[:n], v.reshape(-1)[:n], BETAS, EPS, lr, wd, t)
            close_param(x.reshape(-1), want, update, before[k].reshape(-1), torch.float32, f"step {t}")
    assert opt.t == 3 and lr < 0.1
    m, v = opt.moments(0)
    assert m.shape == (33, 20) and bool((v > 0).all())
    assert not opt.states[2].any()


@pytest.mark.parametrize("bits", [32, 8])
def test_state_dict_goes_on_where_it_was(bits):
    def side():
        g = torch.Generator().manual_seed(1)
        p = torch.randn(50, 60, generator=g).cuda().requires_grad_(True)
        return p, L.AdamW([p], lr=0.05, state_bits=bits, seed=3)

    def steps(p, opt, n):
        for _ in range(n):
            opt.zero_grad()
            (p ** 4).sum().backward()
            opt.step()

    p, opt = side()
    steps(p, opt, 3)
    q, other = side()
    with torch.no_grad():
        q.copy_(p)
    other.load_state_dict(opt.state_dict())
    steps(p, opt, 2)
    steps(q, other, 2)
    assert torch.equal(p, q) and opt.t == other.t == 5
    wrong = L.AdamW([torch.ones(3, device="cuda")], state_bits=bits)
    with pytest.raises(ValueError, match="another"):
        wrong.load_state_dict(opt.state_dict())
    with pytest.raises(ValueError, match="no AdamW"):
        wrong.load_state_dict({})


def test_refusals():
    p, s, step = torch.ones(8, device="cuda"), layers.adamw_state(torch.ones(8, device="cuda")), torch.zeros(2, dtype=torch.int64, device="cuda")
    for call in (lambda: layers.adamw_step([p], [p], [], step, lr=1.0), lambda: layers.adamw_step([p], [p.cpu()], [s], step, lr=1.0),
                 lambda: layers.adamw_step([p], [p[:4]], [s], step, lr=1.0), lambda: layers.adamw_step([p], [p], [s[:8]], step, lr=1.0),
                 lambda: layers.adamw_step([p], [p], [s], step[:1], lr=1.0), lambda: layers.adamw_step([p], [p], [s], step.int(), lr=1.0),
                 lambda: layers.adamw_step([p], [p], [s], step, lr=1.0, state_bits=8),
                 lambda: layers.adamw_step([p], [p], [s], step, lr=[1.0, 2.0]), lambda: layers.adamw_step([p[::2]], [None], [s], step, lr=1.0),
                 lambda: layers.adamw_step([p.double()], [None], [s], step, lr=1.0),
                 lambda: layers.adamw_step([p], [p.long()], [s], step, lr=1.0), lambda: layers.adamw_moments(s, 300),
                 lambda: L.AdamW([{"params": [p], "betas": (0.5, 0.5)}]), lambda: L.AdamW([torch.ones(3)]),
                 lambda: L.AdamW([p]).add_param_group({"params": [s]})):
        with pytest.raises(ValueError):
            call()
    for kw in (dict(betas=(1.0, 0.9)), dict(betas=(0.9, -0.1)), dict(eps=-1.0), dict(lr=float("nan")), dict(weight_decay=float("inf"))):
        with pytest.raises(L.LoptError):
            layers.adamw_step([p], [p.clone()], [s], step, **{"lr": 1.0, **kw})
    with pytest.raises(L.LoptError, match="overlap"):
        layers.adamw_step([p, p], [p.clone(), p.clone()], [s, s.clone()], step, lr=1.0)
    with pytest.raises(L.LoptError, match="overlap"):
        layers.adamw_step([p], [p], [s], step, lr=1.0)
    assert step.tolist() == [0, 0] and bool((p == 1).all())


# ---- 8-bit codes follow from the fp32 moments and the random bits, and from nothing else

def fp32_codes(g, state, seed, t, place):
    """(m, v) in fp32 and the buffer of their codes, each rounded with its random bits alone."""
    m, v, _ = step_moments(g, state, 8, BETAS, seed, t, place)
    r = random_bits(seed, t, place, 0, m.size).reshape(m.shape)
    cm, em = encode(m.astype(np.float64), 15, (r & np.uint64(0xFFFF)).astype(np.float64) / 65536)
    cv, ev = encode(v.astype(np.float64), 31, (r >> np.uint64(16)).astype(np.float64) / 65536)
    new = np.zeros((len(m), 2 * BLOCK + 16), np.uint8)
    new[:, :BLOCK] = np.where((em == 255)[:, None], 0, cm + 128 * ((m < 0) & (cm > 0)))
    new[:, BLOCK:2 * BLOCK] = np.where((ev == 255)[:, None], 0, np.where((v > 0) & (cv == 0), 1, cv))
    new[:, 2 * BLOCK], new[:, 2 * BLOCK + 1] = em, ev
    return m, v, new.reshape(-1)


def step8_and_check(ps, gs, states, step, lr, wd, seed, what):
    lrs, wds = (np.broadcast_to(np.asarray(v, np.float64), len(ps)) for v in (lr, wd))
    before = [as_numpy(p).reshape(-1).copy() for p in ps], [as_numpy(s).copy() for s in states]
    layers.adamw_step(ps, gs, states, step, lr=lr, betas=BETAS, eps=EPS, weight_decay=wd, state_bits=8, seed=seed)
    t = int(step[0])
    for k, (p, g) in enumerate(zip(ps, gs)):
        if g is None:
            assert np.array_equal(as_numpy(p).reshape(-1), before[0][k]) and np.array_equal(as_numpy(states[k]), before[1][k])
            continue
        m, v, new = fp32_codes(as_numpy(g).reshape(-1), before[1][k], seed, t, k)
        off = np.count_nonzero(as_numpy(states[k]) != new)
        assert off == 0, f"{what} tensor {k}: {off} codes differ"
        n = p.numel()
        want, update = step_param(before[0][k], m.reshape(-1)[:n], v.reshape(-1)[:n], BETAS, EPS, lrs[k], wds[k], t)
        close_param(p.reshape(-1), want, update, before[0][k], p.dtype, f"{what} tensor {k}")


@pytest.mark.parametrize("gt", TYPES, ids=str)
@pytest.mark.parametrize("pt", TYPES, ids=str)
def test_codes_of_the_fp32_moments(pt, gt):
    ps, gs, states = make(SIZES, pt, gt, 8, 3)
    step = torch.zeros(2, dtype=torch.int64, device="cuda")
    for t in range(3):
        step8_and_check(ps, gs, states, step, 1e-2, 0.1, 77, f"step {t}")
        gs = [g.flip(0) * 0.5 for g in gs]


def test_codes_of_the_fp32_moments_over_a_long_list():
    g = torch.Generator().manual_seed(9)
    sizes = torch.randint(1, 3000, (391,), generator=g).tolist()
    ps, gs, states = [], [], []
    for k, n in enumerate(sizes):
        p, d, s = make([n], TYPES[k % 3], TYPES[0 if k % 2 else k % 3], 8, k)
        ps, gs, states = ps + p, gs + ([None] if k % 7 == 3 else d), states + s
    lr, wd = (1e-2 * torch.rand(391, generator=g)).tolist(), (0.2 * torch.rand(391, generator=g)).tolist()
    step = torch.zeros(2, dtype=torch.int64, device="cuda")
    for t in range(2):
        step8_and_check(ps, gs, states, step, lr, wd, 5, f"step {t}")


def test_codes_and_parameters_of_two_steps_of_many_elements():
    """2^24 elements of one size, some of whose v lie on a code's border in fp32 alone: every code of two steps, and every
    parameter, which the second step moves by what the first one kept."""
    n = 1 << 24
    g = torch.Generator().manual_seed(21)
    ps, gs = [0.1 * torch.randn(n, generator=g).cuda()], [1e-3 * torch.randn(n, generator=g).cuda()]
    states, step = [layers.adamw_state(ps[0], 8)], torch.zeros(2, dtype=torch.int64, device="cuda")
    for t in range(2):
        step8_and_check(ps, gs, states, step, 1e-3, 0.1, 5, f"step {t}")
        gs = [g.flip(0) for g in gs]


def test_codes_below_the_least_exponent():
    """2^24 elements over five decades, many of them below their block's least exponent, where a scaled number loses bits: the
    random bits meet what is there of it and not what it was rounded up to."""
    n = 1 << 24
    ps, gs, states = make([n], torch.float32, torch.float32, 8, 21)
    step = torch.zeros(2, dtype=torch.int64, device="cuda")
    for t in range(2):
        step8_and_check(ps, gs, states, step, 1e-3, 0.1, 5, f"step {t}")
        gs = [g.flip(0) for g in gs]
