"""The embedding and its gradient on the GPU against their definitions in 64 bits."""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - CPU container
    pytest.skip("no GPU", allow_module_level=True)

from learned_optimizer_step_amd import layers  # noqa: E402
from learned_optimizer_step_amd import lopt as L  # noqa: E402
from ops_cases import CODE, TYPES, U, close, rounding  # noqa: E402

# (tokens, rows, columns): the sort's passes (rows below and from 256, 65536), its tiles of 1024 tokens and its one-block
# limit of 8192, chunks that end inside runs, widths around the slabs of 64 vectors
SHAPES = [(1, 1, 1), (1, 7, 5), (3, 2, 64), (77, 1000, 65), (8, 255, 33), (64, 256, 8), (500, 257, 130), (4095, 300, 17),
          (4096, 65535, 20), (4097, 65536, 12), (9000, 70001, 8), (1024, 3, 257), (2000, 50257, 40), (5000, 1, 70),
          (16384, 500, 12), (16385, 500, 12), (40000, 1000, 36), (333, 40, 513), (333, 40, 1030), (50, 20, 2048),
          # a handful of tokens in one launch; tables of 16 MB and more, whose rows are cleared in several launches
          (64, 30, 3), (65, 9, 70), (128, 50, 515), (129, 50, 515), (5, 50257, 130), (700, 50257, 130), (6000, 33000, 257),
          (20000, 40000, 131), (9000, 100, 3)]


def make_ids(n, rows, seed, kind):
    g = torch.Generator().manual_seed(seed)
    if kind == "text":
        ids = (torch.exp(torch.rand(n, generator=g) * math.log(rows + 1)).long() - 1).clamp(0, rows - 1)
    elif kind == "one":
        ids = torch.full((n,), rows - 1)
    else:
        ids = torch.randint(0, rows, (n,), generator=g)
    bad = torch.rand(n, generator=g) < 0.15
    ids[bad] = torch.tensor([-1, -7, rows, rows + 1000, 2 ** 31 - 1, -2 ** 31])[torch.randint(0, 6, (int(bad.sum()),), generator=g)]
    return ids


def dense(dout, ids, rows, scale, row0=0):
    """(gradient, what its terms add up to without signs, tokens of each row)"""
    ids = ids.reshape(-1) - row0
    d = dout.reshape(ids.numel(), -1).double() * scale
    there = (ids >= 0) & (ids < rows)
    out, size = torch.zeros(2, rows, d.shape[1], dtype=torch.float64)
    out.index_add_(0, ids[there], d[there])
    size.index_add_(0, ids[there], d[there].abs())
    return out, size, torch.bincount(ids[there], minlength=rows)


@pytest.mark.parametrize("t", TYPES, ids=str)
@pytest.mark.parametrize("n,rows,cols", SHAPES)
def test_against_the_definition(n, rows, cols, t):
    g = torch.Generator().manual_seed(n + rows)
    scale = math.sqrt(cols)
    w = torch.randn(rows, cols, generator=g)
    for kind, idt in (("text", torch.int64), ("one", torch.int32), ("any", torch.int32)):
        ids = make_ids(n, rows, n + cols, kind)
        wt = torch.float32 if kind != "any" else t
        out = layers.embedding_forward(ids.to(idt).cuda(), w.to(wt).cuda(), scale, dtype=t)
        there = (ids >= 0) & (ids < rows)
        want = w.to(wt).double()[ids.clamp(0, rows - 1)] * torch.tensor(scale, dtype=torch.float32).double() * there[:, None]
        # the product in fp32, then the type's rounding
        close(out, want, rounding(want, t) + 2 * U * want.abs(), "out")
        dout = torch.randn(n, cols, generator=g).to(t)
        dw = layers.embedding_backward(dout.cuda(), ids.to(idt).cuda(), rows, scale, dtype=wt)
        want, size, count = dense(dout, ids, rows, torch.tensor(scale, dtype=torch.float32).double())
        # a term passes at most its row's tokens' additions, and the product
        close(dw, want, rounding(want, wt) + (count[:, None] + 2) * U * size, "dw")
        filled = torch.full((rows, cols), math.nan, dtype=wt, device="cuda")     # whatever was there
        assert torch.equal(dw, layers.embedding_backward(dout.cuda(), ids.to(idt).cuda(), rows, scale, out=filled))


def test_long_runs_of_one_row():
    """Runs over many chunks: ones add up exactly in fp32 in any order; random values give the same bits again."""
    for n in (9, 40, 3000, 20000):
        ids = torch.zeros(n, dtype=torch.int64)
        ids[1::3] = 5
        dw = layers.embedding_backward(torch.ones(n, 40).cuda(), ids.cuda(), 9)
        want = torch.bincount(ids, minlength=9).float()
        assert torch.equal(dw.cpu(), want[:, None].expand(-1, 40))
        d = torch.randn(n, 40, generator=torch.Generator().manual_seed(n)).cuda()
        assert torch.equal(layers.embedding_backward(d, ids.cuda(), 9), layers.embedding_backward(d, ids.cuda(), 9))


def test_a_shard_of_the_table_and_rows_left_alone():
    n, rows, cols = 600, 40, 50
    g = torch.Generator().manual_seed(3)
    ids = torch.randint(0, 3 * rows, (4, n // 4), generator=g).cuda()
    w = torch.randn(3 * rows, cols, generator=g).cuda()
    dout = torch.randn(4, n // 4, cols, generator=g).cuda()
    whole, gw = layers.embedding_forward(ids, w, 2.0), layers.embedding_backward(dout, ids, 3 * rows, 2.0)
    outs = [layers.embedding_forward(ids, w[k * rows:(k + 1) * rows], 2.0, row0=k * rows) for k in range(3)]
    assert torch.equal(sum(outs), whole) and whole.shape == (4, n // 4, cols)
    parts = [layers.embedding_backward(dout, ids, rows, 2.0, row0=k * rows) for k in range(3)]
    assert torch.equal(torch.cat([(p != 0).any(1) for p in parts]), (gw != 0).any(1))
    # the same sums up to the chunks' borders
    size = dense(dout.cpu(), ids.cpu(), 3 * rows, 2.0)[1]
    close(torch.cat(parts), gw.double().cpu(), 2 * 40 * U * size, "shards")
    far = 1 << 40
    assert torch.equal(layers.embedding_forward(ids + far, w, 2.0, row0=far), whole)


@pytest.mark.parametrize("n", [1, 100, 700, 9000])
@pytest.mark.parametrize("gt", TYPES, ids=str)
def test_accumulating(gt, n):
    rows, cols = 5000, 72
    g = torch.Generator().manual_seed(4)
    ids = make_ids(n, rows, 9, "text").cuda()
    dout = torch.randn(n, cols, generator=g).bfloat16().cuda()
    base = torch.randn(rows, cols, generator=g).to(gt).cuda()
    base[17] = float("nan")     # a row that no token names keeps its bits
    ids[ids == 17] = 18
    out = base.clone()
    assert layers.embedding_backward(dout, ids, rows, 0.5, out=out, accumulate=True) is out
    named = torch.zeros(rows, dtype=torch.bool)
    named[ids[(ids >= 0) & (ids < rows)].cpu()] = True
    assert torch.equal(out.view(torch.int16 if gt != torch.float32 else torch.int32)[~named.cuda()],
                       base.view(torch.int16 if gt != torch.float32 else torch.int32)[~named.cuda()])
    want, size, count = dense(dout.cpu(), ids.cpu(), rows, 0.5)
    want = (want + base.double().cpu())[named]
    close(out[named.cuda()], want, rounding(want, gt) + (count[named][:, None] + 3) * U * (size[named] + want.abs()), "added")


def test_strides_and_what_lies_around():
    n, rows, cols, ld = 300, 60, 37, 50
    g = torch.Generator().manual_seed(6)
    ids = make_ids(n, rows, 1, "any").cuda()
    for t in TYPES:
        big = torch.randn(rows, ld, generator=g).to(t).cuda()
        dbig = torch.randn(n, ld, generator=g).to(t).cuda()
        w, d = big[:, 3:3 + cols], dbig[:, 1:1 + cols]
        assert torch.equal(layers.embedding_forward(ids, w, 1.5), layers.embedding_forward(ids, w.contiguous(), 1.5))
        dw = layers.embedding_backward(d.contiguous(), ids, rows, 1.5, dtype=t)
        assert torch.equal(layers.embedding_backward(d, ids, rows, 1.5, dtype=t), dw)
        out = torch.full((rows + 1, ld), 3.0, dtype=t, device="cuda")
        nb = L.lopt_embedding_backward_workspace(n, rows, cols)
        ws = torch.full((nb + 256,), 171, dtype=torch.uint8, device="cuda")   # what was in it does not matter
        code = CODE[t]
        L.lopt_embedding_backward(n, ids.data_ptr(), 8, d.data_ptr(), ld, code, rows, cols, 0, 1.5,
                                  out.data_ptr() + 2 * out.element_size(), ld, code, 0, ws.data_ptr(), nb,
                                  torch.cuda.current_stream().cuda_stream)
        assert torch.equal(out[:rows, 2:2 + cols], dw)
        out[:rows, 2:2 + cols] = 3.0
        assert bool((out == 3.0).all()) and bool((ws[nb:] == 171).all())
    # ids with strides
    two = torch.randint(0, rows, (n, 2), generator=g).cuda()
    w = torch.randn(rows, cols, generator=g).cuda()
    assert torch.equal(layers.embedding_forward(two[:, 1], w), w[two[:, 1]])


def test_infinities_stay_in_their_rows():
    ids = torch.tensor([1, 2, -1, 2, 3]).cuda()
    dout = torch.ones(5, 9).cuda()
    dout[2] = float("nan")          # padding: not read into any row
    dout[3, 4] = float("inf")
    dw = layers.embedding_backward(dout, ids, 5)
    assert not torch.isnan(dw).any() and torch.isinf(dw).nonzero().tolist() == [[2, 4]]
    w = torch.ones(5, 9).cuda()
    w[0] = float("nan")
    out = layers.embedding_forward(torch.tensor([1, -1, 5]).cuda(), w)
    assert out.tolist() == [[1.0] * 9, [0.0] * 9, [0.0] * 9]


def test_no_tokens_and_no_rows():
    none = torch.empty(0, dtype=torch.int64, device="cuda")
    w = torch.randn(5, 8, device="cuda")
    assert layers.embedding_forward(none, w).shape == (0, 8)
    assert not layers.embedding_backward(torch.empty(0, 8, device="cuda"), none, 5).any()
    out = w.clone()
    layers.embedding_backward(torch.empty(0, 8, device="cuda"), none, 5, out=out, accumulate=True)
    assert torch.equal(out, w)
    ids = torch.tensor([0, 3], device="cuda")
    assert not layers.embedding_forward(ids, torch.empty(0, 8, device="cuda")).any()
    assert layers.embedding_backward(w[:2], ids, 0).shape == (0, 8)
    assert not layers.embedding_backward(w[:2], ids - 9, 4).any()


def test_autograd():
    g = torch.Generator().manual_seed(5)
    ids = torch.randint(-1, 30, (6, 20), generator=g).cuda()
    w = torch.randn(30, 48, generator=g).cuda().requires_grad_(True)
    out = layers.embedding(ids, w, 3.0, dtype=torch.bfloat16)
    assert out.dtype == torch.bfloat16 and out.shape == (6, 20, 48)
    d = torch.randn(6, 20, 48, generator=g).bfloat16().cuda()
    grad, = torch.autograd.grad(out, w, d)
    want, size, count = dense(d.cpu(), ids.cpu(), 30, 3.0)
    close(grad, want, rounding(want, torch.float32) + (count[:, None] + 2) * U * size, "grad")
    # linear in w: differences are exact up to roundings
    k = torch.randn(30, 48, generator=g).double()
    f = lambda v: (layers.embedding_forward(ids, v.float().cuda(), 3.0).double().cpu() * d.double().cpu()).sum()  # noqa: E731
    diff = f(w.detach().double().cpu() + k) - f(w.detach().double().cpu())
    assert abs(diff - (grad.double().cpu() * k).sum()) <= 1e-5 * (grad.double().cpu() * k).abs().sum()
    layers.embedding(ids, w, 3.0).sum().backward()     # an expanded gradient
    assert torch.isfinite(w.grad).all()


def test_on_another_stream_and_in_a_graph():
    n, rows, cols = 5000, 300, 100
    g = torch.Generator().manual_seed(12)
    d = torch.randn(n, cols, generator=g).cuda()
    lists = [make_ids(n, rows, k, "text").cuda() for k in range(4)]
    want = layers.embedding_backward(d, lists[0], rows)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = layers.embedding_backward(d, lists[0], rows)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(want, got)
    ids, out, total = lists[0].clone(), torch.empty(rows, cols, device="cuda"), torch.zeros(rows, cols, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layers.embedding_backward(d, ids, rows, out=out)
        layers.embedding_backward(d, ids, rows, out=total, accumulate=True)
    total.zero_()
    sums = torch.zeros_like(total)
    for k, l in enumerate(lists):
        ids.copy_(l)
        eager = layers.embedding_backward(d, l, rows)
        layers.embedding_backward(d, l, rows, out=sums, accumulate=True)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager) and torch.equal(total, sums), k


def test_more_elements_than_32_bits_count():
    rows, cols = (1 << 20) + 5, 2048
    ids = torch.tensor([rows - 1, 3, rows - 1, rows - 2], device="cuda")
    d = torch.randn(4, cols, device="cuda").bfloat16()
    dw = layers.embedding_backward(d, ids, rows, dtype=torch.bfloat16)
    assert torch.equal(dw[-1], (d[0].float() + d[2].float()).bfloat16()) and torch.equal(dw[-2], d[3]) and torch.equal(dw[3], d[1])
    assert int((dw != 0).any(1).sum()) == 3
    assert torch.equal(layers.embedding_forward(ids, dw)[0], dw[-1])


def test_refusals_of_the_tensors():
    w, ids = torch.ones(4, 8, device="cuda"), torch.zeros(3, dtype=torch.int64, device="cuda")
    for call in (lambda: layers.embedding(ids.float(), w), lambda: layers.embedding(ids.cpu(), w),
                 lambda: layers.embedding(ids, w[0]), lambda: layers.embedding(ids, w.double()),
                 lambda: layers.embedding_forward(ids, w, dtype=torch.float64),
                 lambda: layers.embedding_backward(w, ids, 4), lambda: layers.embedding_backward(w[:3], ids, 4, accumulate=True),
                 lambda: layers.embedding_backward(w[:3], ids, 4, out=torch.ones(5, 8, device="cuda"))):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: layers.embedding(ids, w, float("nan")), lambda: layers.embedding(ids, w, row0=-1)):
        with pytest.raises(L.LoptError):
            call()


def test_a_handful_of_tokens_of_more_columns_than_one_grid_has_threads_for():
    """2^34 elements (34 GB in bf16): a wave a token and 256 columns would be 2^32 threads."""
    n, rows, cols = 128, 3, 1 << 27
    d = torch.empty(n, cols, dtype=torch.bfloat16, device="cuda")
    for t in range(n):
        d[t].fill_(float(t % 5 - 2))
    d[7, -1], d[127, 0] = 9.0, -7.0
    ids = torch.arange(n, device="cuda") % 4 - 1      # a quarter of the tokens names no row
    out = torch.full((rows, cols), 3.0, device="cuda")
    layers.embedding_backward(d, ids, rows, 0.5, out=out, accumulate=True)
    for r in range(rows):
        want = 3.0 + 0.5 * sum(t % 5 - 2 for t in range(n) if t % 4 - 1 == r)
        assert bool((out[r, 1:-1] == want).all()), r
        assert out[r, 0] == want + 0.5 * (-7.0 - (127 % 5 - 2)) * (127 % 4 - 1 == r), r
        assert out[r, -1] == want + 0.5 * (9.0 - (7 % 5 - 2)) * (7 % 4 - 1 == r), r


def ids_with_runs(n, rows, chunk, seed):
    """Ids whose sorted runs begin and end 0, 1, 7, 8, 9 and 10 tokens behind borders of chunks, near ones and far ones, in
    any order; every 20th token names no row."""
    g = torch.Generator().manual_seed(seed)
    named, at, counts = n - n // 20, 0, []
    while at < named and len(counts) < rows - 1:
        k = len(counts)
        ahead = 300 if k % 50 == 25 else (0, 1, 1, 2, 3, 1, 6)[k % 7]
        end = (at // chunk + ahead) * chunk + (0, 1, 7, 8, 9, 10, 8, 9)[k % 8]
        end = min(named, end if end > at else at + 1 + k % 3)
        counts.append(end - at)
        at = end
    counts.append(named - at)
    which = torch.randperm(rows, generator=g)[:len(counts)].sort().values
    ids = torch.cat([which.repeat_interleave(torch.tensor(counts)), torch.full((n - named,), -1)])
    return ids[torch.randperm(n, generator=g)]


@pytest.mark.parametrize("n,rows,cols,chunk", [
    (8192, 3000, 40, 8), (8193, 3000, 40, 8), (16383, 60000, 5, 8),          # the longest list of one block, and the next
    (65535, 5000, 30, 8), (65536, 5000, 30, 16), (131072, 9000, 9, 32), (196608, 9000, 64, 48), (196608, 9000, 3, 48),
    (13120, 700, 1040, 16), (26240, 1000, 1037, 32), (39360, 1500, 1040, 48),   # several slabs
    (262145, 200, 8, 48), (300001, 40000, 6, 48), (1100003, 300, 4, 48),     # blocks of the sort that take more than one tile
    (9000, (1 << 24) + 5, 2, 8), (70000, (1 << 24) + 5, 1, 16), (8000, (1 << 24) + 5, 1, 8)])   # four passes
@pytest.mark.parametrize("dt,gt", [(torch.bfloat16, torch.float32), (torch.float32, torch.float32), (torch.float16, torch.bfloat16)],
                         ids=str)
def test_the_geometry_of_long_lists(n, rows, cols, chunk, dt, gt):
    """Whole numbers, whose sums are exact in fp32 in any order, for every length of a chunk."""
    slabs = (cols + 255) // 256
    assert chunk == max([8] + [c for c in (16, 32, 48) if n // c * slabs >= 4096])
    ids = ids_with_runs(n, rows, chunk, n)
    g = torch.Generator().manual_seed(cols)
    d = torch.randint(-8, 9, (n, cols), generator=g).to(dt)
    there = ids >= 0
    want = torch.zeros(rows, cols, dtype=torch.float64).index_add_(0, ids[there], d[there].double())
    assert want.abs().max() < 2 ** 24
    base = torch.randint(-8, 9, (rows, cols), generator=g).to(gt)
    ids, d = ids.cuda(), d.cuda()
    out = torch.full((rows, cols), math.nan, dtype=gt, device="cuda")
    assert torch.equal(layers.embedding_backward(d, ids, rows, out=out).cpu(), want.float().to(gt))
    # one rounding of the sum, and rows that no token names as they were
    added = layers.embedding_backward(d, ids, rows, out=base.cuda(), accumulate=True)
    assert torch.equal(added.cpu(), (want + base.double()).float().to(gt))
