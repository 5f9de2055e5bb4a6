"""The residual update's calls on the CPU: workspace sizes and every refusal.  Addresses are made up and never read."""
import pytest
import torch

from learned_optimizer_step_amd import lopt as L

A = [(k + 1) << 40 for k in range(20)]
BAD, UNSUPPORTED, WORKSPACE = L.LOPT_ERR_INVALID_ARGUMENT, L.LOPT_ERR_UNSUPPORTED, L.LOPT_ERR_WORKSPACE

FWD = dict(kind=0, post=1, pre=1, rows=5, cols=16, dtype=1, x=A[0], ldx=16, y=A[1], ldy=16, gate_kind=1, gate=A[2], ldg=0,
           post_weight=A[3], post_bias=A[4], weight=A[5], bias=A[6], w_dtype=0, alpha=1.0, beta=1.0, eps=1e-5, h=A[7], ldh=16, z=A[8],
           ldz=16, stats=A[9], stream=None)
BWD = dict(kind=0, post=1, pre=1, rows=5, cols=16, dtype=1, dh=A[0], lddh=16, dz=A[1], lddz=16, y=A[2], ldy=16, h=A[3], ldh=16,
           stats=A[4], gate_kind=1, gate=A[5], ldg=0, post_weight=A[6], post_bias=A[7], weight=A[8], w_dtype=0, alpha=1.0, beta=1.0,
           dx=A[9], lddx=16, dy=A[10], lddy=16, dgate=A[11], lddg=0, dpost_weight=A[12], dpost_bias=A[13], dweight=A[14], dbias=A[15],
           g_dtype=0, accumulate=0, workspace=A[16], ws_bytes=1 << 30, stream=None)

CASES = [
    *[("lopt_residual_norm_forward", FWD, c, s) for c, s in [
        (dict(kind=2), BAD), (dict(post=0, pre=0), BAD), (dict(rows=-1), BAD), (dict(cols=0), BAD), (dict(rows=1 << 31), UNSUPPORTED),
        (dict(dtype=3), BAD), (dict(w_dtype=7), BAD), (dict(x=None), BAD), (dict(y=None), BAD), (dict(h=None), BAD), (dict(z=None), BAD),
        (dict(ldx=15), BAD), (dict(ldy=15), BAD), (dict(ldh=15), BAD), (dict(ldz=3), BAD), (dict(gate_kind=3), BAD), (dict(gate_kind=-1), BAD),
        (dict(gate=None), BAD), (dict(gate_kind=2, ldg=15), BAD), (dict(gate=A[2] + 2), UNSUPPORTED), (dict(x=A[0] + 1), UNSUPPORTED),
        (dict(eps=-1.0), BAD), (dict(eps=float("nan")), BAD), (dict(alpha=float("inf")), BAD), (dict(beta=float("nan")), BAD),
        (dict(kind=1), BAD), (dict(kind=1, bias=None), BAD), (dict(post=0), BAD), (dict(post=0, post_weight=None), BAD), (dict(pre=0), BAD),
        (dict(pre=0, weight=None, bias=None), BAD), (dict(h=A[0]), BAD), (dict(z=A[7]), BAD), (dict(h=A[1] + 32), BAD), (dict(stats=A[8] + 4), BAD),
        (dict(stats=A[9] + 2), UNSUPPORTED), (dict(weight=A[7]), BAD), (dict(ldx=1 << 60), UNSUPPORTED)]],
    *[("lopt_residual_norm_backward", BWD, c, s) for c, s in [
        (dict(kind=-1), BAD), (dict(post=0, pre=0), BAD), (dict(rows=-2), BAD), (dict(cols=0), BAD), (dict(dtype=9), BAD), (dict(g_dtype=5), BAD),
        (dict(w_dtype=5), BAD), (dict(y=None), BAD), (dict(h=None), BAD), (dict(stats=None), BAD), (dict(kind=1), BAD),
        (dict(kind=1, post_bias=None, dpost_bias=None), BAD), (dict(post=0), BAD), (dict(pre=0), BAD), (dict(pre=0, weight=None, dweight=None, dbias=None), BAD),
        (dict(gate_kind=0), BAD), (dict(gate=None), BAD), (dict(lddh=0), BAD), (dict(lddx=3), BAD), (dict(gate_kind=2, ldg=16, lddg=2), BAD),
        (dict(dx=A[0]), BAD), (dict(dy=A[9]), BAD), (dict(dgate=A[14] + 4), BAD), (dict(workspace=None), WORKSPACE), (dict(ws_bytes=4), WORKSPACE),
        (dict(workspace=A[16] + 128), WORKSPACE), (dict(workspace=A[9]), BAD), (dict(dweight=A[14] + 2), UNSUPPORTED),
        (dict(alpha=float("nan")), BAD), (dict(beta=float("inf")), BAD)]],
]


@pytest.fixture(scope="module", autouse=True)
def lib():
    import os
    if not os.path.exists(L.LIB_PATH):
        pytest.skip("liblopt.so not built")


@pytest.mark.parametrize("k", range(len(CASES)), ids=lambda k: f"{CASES[k][0][19:]}-{CASES[k][2]}")
def test_refusals(k):
    call, args, change, status = CASES[k]
    with pytest.raises(L.LoptError) as e:
        getattr(L, call)(*{**args, **change}.values())
    assert e.value.status == status, e.value
    assert len(str(e.value)) > 12


def test_workspace_sizes():
    assert L.lopt_residual_norm_backward_workspace(0, 768) == 0
    for rows, cols in ((1, 1), (1, 768), (4096, 1024), (65536, 2048), (1 << 30, 7), (3, 100_000)):
        b = L.lopt_residual_norm_backward_workspace(rows, cols) - (8 * rows if cols > 8192 else 0)
        # five floats a column and block, of which there are never more than rows or 2048
        assert b % (20 * cols) == 0 and 1 <= b // (20 * cols) <= min(rows, 2048), (rows, cols, b)
    for args in ((-1, 4), (4, 0)):
        with pytest.raises(L.LoptError) as e:
            L.lopt_residual_norm_backward_workspace(*args)
        assert e.value.status == BAD
    assert L.load_library().lopt_residual_norm_backward_workspace(4, 4, None) == BAD


def test_empty_calls_need_no_buffers():
    L.lopt_residual_norm_forward(*{**FWD, "rows": 0, "x": None, "y": None, "h": None, "z": None, "gate": None, "stats": None}.values())
    L.lopt_residual_norm_backward(*{**BWD, "rows": 0, "y": None, "h": None, "dx": None, "dy": None, "dgate": None, "dpost_weight": None,
                                    "dpost_bias": None, "dweight": None, "dbias": None, "gate": None, "stats": None}.values())


def test_no_cpu_path():
    from learned_optimizer_step_amd import layers
    x = torch.ones(3, 8)
    for call in (lambda: layers.residual_norm(x, x), lambda: layers.residual_norm_forward(x, x),
                 lambda: layers.residual_norm_backward(x, x, x, x, torch.ones(4, 3))):
        with pytest.raises(ValueError, match="GPU"):
            call()


def test_room_for_long_rows():
    """Rows over 8192 columns: five floats a column for each of up to 64 blocks, and, of more rows, four floats a row."""
    for rows, cols in ((1, 8193), (64, 9000), (65, 8200), (20481, 8193), (1_000_000, 10_000)):
        b = L.lopt_residual_norm_backward_workspace(rows, cols)
        need = 20 * cols * min(rows, 64) + (16 * rows if rows > 64 else 0)
        assert need <= b < need + 20 * cols + 8 * rows + 1, (rows, cols, b, need)
