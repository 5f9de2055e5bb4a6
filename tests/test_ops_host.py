"""The norm, embedding and distillation calls on the CPU: sizes of workspaces and
every refusal.  Addresses are made up and never read: validation comes first."""
import ctypes

import pytest
import torch

from learned_optimizer_step_amd import lopt as L

A = [(k + 1) << 40 for k in range(12)]   # addresses far apart, 256-byte aligned
BAD, UNSUPPORTED, WORKSPACE = L.LOPT_ERR_INVALID_ARGUMENT, L.LOPT_ERR_UNSUPPORTED, L.LOPT_ERR_WORKSPACE

NORM_FWD = dict(kind=0, rows=5, cols=16, dtype=1, x=A[0], ldx=16, weight=A[1], bias=A[2], w_dtype=0, eps=1e-5, y=A[3], ldy=16,
                mean=A[4], rstd=A[5], stream=None)
NORM_BWD = dict(kind=0, rows=5, cols=16, dtype=1, dy=A[0], lddy=16, x=A[1], ldx=16, weight=A[2], w_dtype=0, mean=A[3],
                rstd=A[4], dx=A[5], lddx=16, dweight=A[6], dbias=A[7], g_dtype=0, accumulate=0, workspace=A[8],
                ws_bytes=1 << 30, stream=None)
EMB_FWD = dict(n_ids=7, ids=A[0], id_bytes=8, rows=10, cols=16, row0=0, table=A[1], ldt=16, t_dtype=0, scale=1.0, out=A[2],
               ldo=16, o_dtype=1, stream=None)
EMB_BWD = dict(n_ids=7, ids=A[0], id_bytes=8, dout=A[1], ldd=16, d_dtype=1, rows=10, cols=16, row0=0, scale=1.0, dtable=A[2],
               ldt=16, g_dtype=0, accumulate=0, workspace=A[3], ws_bytes=1 << 30, stream=None)
DIS_FWD = dict(rows=5, cols=100, dtype=1, logits=A[0], ldz=100, top=4, ids=A[1], ldi=4, id_bytes=8, teacher=A[2], ldu=4,
               u_dtype=0, temperature=2.0, loss=A[3], lse=A[4], stream=None)
DIS_BWD = dict(rows=5, cols=100, dtype=1, dloss=A[0], dloss_stride=1, logits=A[1], ldz=100, top=4, ids=A[2], ldi=4, id_bytes=8,
               teacher=A[3], ldu=4, u_dtype=0, temperature=2.0, lse=A[4], dlogits=A[5], lddz=100, stream=None)

CASES = [
    # (call, its arguments, what is changed, the status)
    *[("lopt_norm_forward", NORM_FWD, c, s) for c, s in [
        (dict(kind=2), BAD), (dict(rows=-1), BAD), (dict(cols=0), BAD), (dict(rows=1 << 31), UNSUPPORTED),
        (dict(cols=1 << 31), UNSUPPORTED), (dict(dtype=3), BAD), (dict(w_dtype=-1), BAD), (dict(x=None), BAD),
        (dict(y=None), BAD), (dict(ldx=15), BAD), (dict(ldy=15), BAD), (dict(x=A[0] + 1), UNSUPPORTED),
        (dict(weight=A[1] + 2), UNSUPPORTED), (dict(eps=-1.0), BAD), (dict(eps=float("nan")), BAD),
        (dict(eps=float("inf")), BAD), (dict(kind=1), BAD), (dict(kind=1, bias=None), BAD), (dict(y=A[0]), BAD),
        (dict(y=A[0] + 2 * 16 * 4), BAD), (dict(mean=A[3] + 8), BAD), (dict(rstd=A[4] + 16), BAD),
        (dict(ldx=1 << 59), UNSUPPORTED), (dict(mean=A[4] + 2), UNSUPPORTED)]],
    *[("lopt_norm_backward", NORM_BWD, c, s) for c, s in [
        (dict(kind=-1), BAD), (dict(rows=-2), BAD), (dict(cols=0), BAD), (dict(dtype=9), BAD), (dict(g_dtype=5), BAD),
        (dict(dy=None), BAD), (dict(x=None), BAD), (dict(mean=None), BAD), (dict(rstd=None), BAD), (dict(kind=1), BAD),
        (dict(kind=1, mean=None), BAD), (dict(lddy=0), BAD), (dict(lddx=3), BAD), (dict(dx=A[0]), BAD), (dict(dx=A[1]), BAD),
        (dict(dbias=A[6] + 4), BAD), (dict(workspace=None), WORKSPACE), (dict(ws_bytes=4), WORKSPACE),
        (dict(workspace=A[8] + 128), WORKSPACE), (dict(workspace=A[6]), BAD), (dict(dweight=A[6] + 2), UNSUPPORTED)]],
    *[("lopt_embedding_forward", EMB_FWD, c, s) for c, s in [
        (dict(n_ids=-1), BAD), (dict(n_ids=(1 << 27) + 1), UNSUPPORTED), (dict(ids=None), BAD), (dict(id_bytes=2), BAD),
        (dict(rows=-1), BAD), (dict(cols=0), BAD), (dict(rows=1 << 31), UNSUPPORTED), (dict(row0=-1), BAD),
        (dict(cols=(1 << 30) + 1, ldt=1 << 31, ldo=1 << 31), UNSUPPORTED),
        (dict(row0=(1 << 40) + 1), BAD), (dict(table=None), BAD), (dict(ldt=8), BAD), (dict(t_dtype=4), BAD),
        (dict(o_dtype=4), BAD), (dict(scale=float("inf")), BAD), (dict(out=None), BAD), (dict(out=A[1] + 64), BAD),
        (dict(ldo=15), BAD), (dict(ids=A[0] + 4), UNSUPPORTED)]],
    *[("lopt_embedding_backward", EMB_BWD, c, s) for c, s in [
        (dict(n_ids=-1), BAD), (dict(n_ids=(1 << 27) + 1), UNSUPPORTED), (dict(ids=None), BAD), (dict(id_bytes=1), BAD),
        (dict(dout=None), BAD), (dict(ldd=2), BAD), (dict(d_dtype=3), BAD), (dict(dtable=None), BAD), (dict(ldt=1), BAD),
        (dict(g_dtype=3), BAD), (dict(row0=-5), BAD), (dict(scale=float("nan")), BAD), (dict(dtable=A[1]), BAD),
        (dict(workspace=None), WORKSPACE), (dict(ws_bytes=100), WORKSPACE), (dict(workspace=A[3] + 4), WORKSPACE),
        (dict(workspace=A[2]), BAD)]],
    *[("lopt_distill_forward", DIS_FWD, c, s) for c, s in [
        (dict(rows=-1), BAD), (dict(cols=0), BAD), (dict(dtype=3), BAD), (dict(logits=None), BAD), (dict(ldz=99), BAD),
        (dict(top=0), BAD), (dict(top=1025, ldi=1025, ldu=1025), UNSUPPORTED), (dict(ids=None), BAD), (dict(ldi=3), BAD),
        (dict(id_bytes=0), BAD), (dict(teacher=None), BAD), (dict(ldu=1), BAD), (dict(u_dtype=7), BAD),
        (dict(temperature=0.0), BAD), (dict(temperature=-1.0), BAD), (dict(temperature=float("nan")), BAD),
        (dict(temperature=float("inf")), BAD), (dict(temperature=1e-45), BAD), (dict(loss=A[0]), BAD),
        (dict(lse=A[3] + 4), BAD)]],
    *[("lopt_distill_backward", DIS_BWD, c, s) for c, s in [
        (dict(rows=-1), BAD), (dict(dloss=None), BAD), (dict(dloss_stride=-1), BAD), (dict(dloss_stride=1 << 28), BAD),
        (dict(lse=None), BAD), (dict(dlogits=None), BAD), (dict(lddz=99), BAD), (dict(dlogits=A[1] + 2), BAD),
        (dict(dlogits=A[1], lddz=101), BAD), (dict(dlogits=A[3]), BAD), (dict(top=1025, ldi=1025, ldu=1025), UNSUPPORTED),
        (dict(temperature=0.0), BAD), (dict(teacher=None), BAD), (dict(logits=None), BAD)]],
]


@pytest.fixture(scope="module")
def lib():
    import os
    if not os.path.exists(L.LIB_PATH):
        pytest.skip("liblopt.so not built")
    return L.load_library()


@pytest.mark.parametrize("k", range(len(CASES)), ids=lambda k: f"{CASES[k][0][5:]}-{CASES[k][2]}")
def test_refusals(lib, k):
    call, args, change, status = CASES[k]
    with pytest.raises(L.LoptError) as e:
        getattr(L, call)(*{**args, **change}.values())
    assert e.value.status == status, e.value
    assert len(str(e.value)) > 12


def test_workspace_sizes(lib):
    assert L.lopt_norm_backward_workspace(0, 768) == 0
    # one float a column, gradient and block, of which there are never more than rows or 1024
    for rows, cols in ((1, 1), (1, 768), (4096, 1024), (65536, 2048), (1 << 30, 7), (3, 100_000)):
        b = L.lopt_norm_backward_workspace(rows, cols)
        assert b % (8 * cols) == 0 and 1 <= b // (8 * cols) <= min(rows, 1024), (rows, cols, b)
    assert L.lopt_embedding_backward_workspace(0, 10, 16) > 0
    last = 0
    for n in (1, 177, 4096, 65536, 1 << 20, 1 << 27):
        b = L.lopt_embedding_backward_workspace(n, 32000, 64)
        assert b % 256 == 0 and b > last and b >= 16 * n
        last = b
    for call, args in (("lopt_norm_backward_workspace", (-1, 4)), ("lopt_norm_backward_workspace", (4, 0)),
                       ("lopt_embedding_backward_workspace", (-1, 4, 4)), ("lopt_embedding_backward_workspace", (4, -4, 4))):
        with pytest.raises(L.LoptError) as e:
            getattr(L, call)(*args)
        assert e.value.status == BAD
    assert lib.lopt_norm_backward_workspace(4, 4, None) == BAD
    assert lib.lopt_embedding_backward_workspace(4, 4, 4, None) == BAD


def test_empty_calls_need_no_buffers(lib):
    """No rows, no ids: nothing is launched or read (there is no GPU here to launch on)."""
    L.lopt_norm_forward(*{**NORM_FWD, "rows": 0, "x": None, "y": None}.values())
    L.lopt_norm_backward(*{**NORM_BWD, "rows": 0, "dweight": None, "dbias": None, "dy": None, "x": None, "dx": None}.values())
    L.lopt_embedding_forward(*{**EMB_FWD, "n_ids": 0, "ids": None, "out": None}.values())
    L.lopt_embedding_backward(*{**EMB_BWD, "n_ids": 0, "ids": None, "dout": None, "accumulate": 1}.values())
    L.lopt_embedding_backward(*{**EMB_BWD, "rows": 0, "dtable": None}.values())
    L.lopt_distill_forward(*{**DIS_FWD, "rows": 0, "logits": None, "ids": None, "teacher": None}.values())
    L.lopt_distill_backward(*{**DIS_BWD, "rows": 0, "logits": None, "dlogits": None, "ids": None, "teacher": None}.values())


def test_in_place_gradient_of_logits_is_not_an_overlap(lib):
    # refused for its missing lse only
    with pytest.raises(L.LoptError) as e:
        L.lopt_distill_backward(*{**DIS_BWD, "dlogits": A[1], "lse": None}.values())
    assert "lse is NULL" in str(e.value)


def test_layers_have_no_cpu_path(lib):
    from learned_optimizer_step_amd import layers
    x, ids = torch.ones(3, 8), torch.zeros(3, dtype=torch.int64)
    for call in (lambda: layers.layer_norm(x), lambda: layers.rms_norm(x), lambda: layers.embedding(ids, x),
                 lambda: layers.embedding_backward(x, ids, 4), lambda: layers.distill_loss(x, ids[:, None], x[:, :1]),
                 lambda: layers.norm_backward(x, x, None, None, ids),
                 lambda: layers.distill_backward(x[:, 0], x, ids[:, None], x[:, :1], x[:, 0])):
        with pytest.raises(ValueError, match="GPU"):
            call()
    with pytest.raises(ValueError, match="detach"):
        layers.distill_loss(x, ids[:, None], x[:, :1].clone().requires_grad_(True))


def test_the_struct_free_calls_refuse_what_is_no_number(lib):
    with pytest.raises(ctypes.ArgumentError):
        L.lopt_norm_forward(*{**NORM_FWD, "rows": "5"}.values())


def test_the_torch_calls_run_from_the_library_that_the_steps_run_from(lib, tmp_path):
    """LOPT_LIBRARY names another build: the norms, the embedding and the distillation loss are that one's too."""
    import os
    import shutil
    import subprocess
    import sys
    other = tmp_path / "liblopt_other.so"
    shutil.copy(L.LIB_PATH, other)
    code = """if True:
        from learned_optimizer_step_amd import layers, lopt
        import torch
        try:
            layers.layer_norm(torch.ones(2, 3))
        except ValueError as e:
            assert "GPU" in str(e)
        maps = {l.split()[-1] for l in open("/proc/self/maps") if "liblopt" in l}
        print(sorted(maps))
    """
    env = dict(os.environ, LOPT_LIBRARY=str(other))
    root = os.path.dirname(os.path.dirname(os.path.abspath(L.__file__)))
    out = subprocess.run([sys.executable, "-c", code], env=env, cwd=root, capture_output=True, text=True, timeout=300)
    assert out.returncode == 0, out.stderr
    assert out.stdout.strip() == str([str(other)])


@pytest.mark.parametrize("call,args", [("lopt_distill_forward", DIS_FWD), ("lopt_distill_backward", DIS_BWD)])
@pytest.mark.parametrize("temperature", [2e19, 3e38, 4e-39, 3e-39])
def test_temperatures_whose_factors_are_no_floats(lib, call, args, temperature):
    with pytest.raises(L.LoptError) as e:
        getattr(L, call)(*{**args, "temperature": temperature}.values())
    assert e.value.status == BAD and "temperature" in str(e.value)
