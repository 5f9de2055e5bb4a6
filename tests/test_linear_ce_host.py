"""The linear cross entropy's calls on the CPU: workspace sizes and every refusal.  Addresses are made up and never read."""
import pytest
import torch

from learned_optimizer_step_amd import lopt as L

A = [(k + 1) << 40 for k in range(12)]
BAD, UNSUPPORTED, WORKSPACE = L.LOPT_ERR_INVALID_ARGUMENT, L.LOPT_ERR_UNSUPPORTED, L.LOPT_ERR_WORKSPACE

FWD = dict(rows=5, cols=16, vocab=100, dtype=1, x=A[0], ldx=16, w=A[1], ldw=16, targets=A[2], id_bytes=8, loss=A[3], lse=A[4],
           workspace=A[5], ws_bytes=1 << 30, stream=None)
BWD = dict(rows=5, cols=16, vocab=100, dtype=1, dloss=A[0], dloss_stride=1, x=A[1], ldx=16, w=A[2], ldw=16, targets=A[3], id_bytes=8,
           lse=A[4], dx=A[5], lddx=16, dw=A[6], lddw=16, g_dtype=0, accumulate=0, workspace=A[7], ws_bytes=1 << 30, stream=None)

BOTH = [(dict(rows=-1), BAD), (dict(cols=0), BAD), (dict(vocab=0), BAD), (dict(rows=(1 << 24) + 1), UNSUPPORTED),
        (dict(cols=(1 << 20) + 1), UNSUPPORTED), (dict(vocab=1 << 31), UNSUPPORTED), (dict(vocab=(1 << 31) - 300, rows=1 << 17), UNSUPPORTED),
        (dict(vocab=1 << 15, rows=1 << 24), UNSUPPORTED), (dict(vocab=(1 << 31) - 300, rows=257), UNSUPPORTED), (dict(vocab=1 << 30, rows=1), UNSUPPORTED),
        (dict(dtype=3), BAD), (dict(x=None), BAD), (dict(w=None), BAD), (dict(targets=None), BAD), (dict(ldx=15), BAD), (dict(ldw=3), BAD),
        (dict(id_bytes=2), BAD), (dict(workspace=None), WORKSPACE), (dict(ws_bytes=100), WORKSPACE)]
CASES = [
    *[("lopt_linear_ce_forward", FWD, c, s) for c, s in BOTH + [
        (dict(x=A[0] + 1), UNSUPPORTED), (dict(targets=A[2] + 4), UNSUPPORTED), (dict(loss=A[0]), BAD), (dict(lse=A[3] + 16), BAD), (dict(lse=A[4] + 2), UNSUPPORTED),
        (dict(workspace=A[5] + 64), WORKSPACE), (dict(workspace=A[1]), BAD)]],
    *[("lopt_linear_ce_backward", BWD, c, s) for c, s in BOTH + [
        (dict(dloss=None), BAD), (dict(dloss_stride=-1), BAD), (dict(dloss_stride=1 << 28), BAD), (dict(lse=None), BAD), (dict(lddx=15), BAD),
        (dict(lddw=15), BAD), (dict(g_dtype=3), BAD), (dict(dx=A[1]), BAD), (dict(dw=A[2] + 4), BAD), (dict(dw=A[6] + 2), UNSUPPORTED),
        (dict(workspace=A[7] + 8), WORKSPACE), (dict(workspace=A[6]), BAD), (dict(lse=A[5] + 8), BAD)]],
]


@pytest.fixture(scope="module", autouse=True)
def lib():
    import os
    if not os.path.exists(L.LIB_PATH):
        pytest.skip("liblopt.so not built")


@pytest.mark.parametrize("k", range(len(CASES)), ids=lambda k: f"{CASES[k][0][15:]}-{CASES[k][2]}")
def test_refusals(k):
    call, args, change, status = CASES[k]
    with pytest.raises(L.LoptError) as e:
        getattr(L, call)(*{**args, **change}.values())
    assert e.value.status == status, e.value
    assert len(str(e.value)) > 12


def test_workspace_sizes():
    for size in (L.lopt_linear_ce_forward_workspace, L.lopt_linear_ce_backward_workspace):
        assert size(0, 64, 100, 1) == 0
        for n, d, v, t in ((1, 1, 1, 0), (4096, 1024, 50257, 1), (8192, 2048, 32000, 2), (1 << 24, 8, 300, 1), (3, 1 << 20, 4000, 0)):
            assert size(n, d, v, t) > 0
        for args, status in (((-1, 4, 4, 0), BAD), ((4, 0, 4, 0), BAD), ((4, 4, 0, 0), BAD), ((4, 4, 4, 5), BAD), (((1 << 24) + 1, 4, 4, 0), UNSUPPORTED)):
            with pytest.raises(L.LoptError) as e:
                size(*args)
            assert e.value.status == status
    # the logits of GPT-2 355M's step, 412 MB in bf16, are never there at once
    assert L.lopt_linear_ce_backward_workspace(4096, 1024, 50257, 1) < 412e6
    assert L.load_library().lopt_linear_ce_forward_workspace(1, 1, 1, 0, None) == BAD
    assert L.load_library().lopt_linear_ce_backward_workspace(1, 1, 1, 0, None) == BAD


def test_empty_calls_need_no_buffers():
    L.lopt_linear_ce_forward(*{**FWD, "rows": 0, "x": None, "w": None, "targets": None, "loss": None, "lse": None, "workspace": None}.values())
    L.lopt_linear_ce_backward(*{**BWD, "rows": 0, "x": None, "w": None, "targets": None, "dloss": None, "lse": None, "dx": None, "dw": None,
                                "workspace": None}.values())
    L.lopt_linear_ce_backward(*{**BWD, "dx": None, "dw": None}.values())   # nothing asked for


def test_no_cpu_path():
    from learned_optimizer_step_amd import layers
    x, t = torch.ones(3, 8), torch.zeros(3, dtype=torch.int64)
    for call in (lambda: layers.linear_cross_entropy(x, x, t), lambda: layers.linear_ce_forward(x, x, t),
                 lambda: layers.linear_ce_backward(x[:, 0], x, x, t, x[:, 0])):
        with pytest.raises(ValueError, match="GPU"):
            call()


def test_the_largest_vocabulary():
    """64 entries a block of 256 threads for few rows: 2^24 blocks would be 2^32 threads, one more than a grid has room for."""
    most = (1 << 30) - 64
    assert -(-most // 64) * 256 < 1 << 32 <= -(-(most + 1) // 64) * 256
    for size, call, args in ((L.lopt_linear_ce_forward_workspace, L.lopt_linear_ce_forward, FWD),
                             (L.lopt_linear_ce_backward_workspace, L.lopt_linear_ce_backward, BWD)):
        assert size(1, 64, most, 1) > 0
        for vocab in (most + 1, (1 << 30) - 1):
            for refused in (lambda: size(1, 64, vocab, 1), lambda: call(*{**args, "rows": 1, "cols": 64, "ldx": 64, "ldw": 64, "vocab": vocab}.values())):
                with pytest.raises(L.LoptError, match="2\\^30") as e:
                    refused()
                assert e.value.status == UNSUPPORTED


def test_the_forward_workspace_goes_by_the_tokens():
    """A maximum and a sum for every token and tile of 64 entries or more, x laid out, and at most 128 MiB (or 1024 entries) of the weight."""
    for n, d, v, t in ((1, 64, (1 << 30) - 64, 1), (1, 2048, 1 << 20, 1), (3, 768, 50257, 0), (300, 333, 10007, 2), (257, 100, 1 << 22, 1)):
        dp, s = -(-d // 64) * 64, (4, 2, 2)[t]
        piece = max(128 << 20, 1024 * dp * s)
        assert L.lopt_linear_ce_forward_workspace(n, d, v, t) <= 8 * n * (-(-v // 256) * 4) + n * dp * s + piece + 4 * n + 4096, (n, d, v, t)
