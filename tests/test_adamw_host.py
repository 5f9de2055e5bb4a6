"""AdamW's calls on the CPU: sizes of moments and every refusal (addresses are made up and never read), and the definition
that the GPU tests use."""
import numpy as np
import pytest

from adamw_cases import BLOCK, decode, encode, step_moments
from learned_optimizer_step_amd import lopt as L

BAD, UNSUPPORTED = L.LOPT_ERR_INVALID_ARGUMENT, L.LOPT_ERR_UNSUPPORTED
K = 1 << 40
TENSOR = dict(param=K, grad=2 * K, state=3 * K, n=1000, lr=1e-3, weight_decay=0.0, p_dtype=0, g_dtype=0)
CALL = dict(state_bits=32, beta1=0.9, beta2=0.999, eps=1e-8, seed=0, step=9 * K, stream=None)


@pytest.fixture(scope="module", autouse=True)
def lib():
    import os
    if not os.path.exists(L.LIB_PATH):
        pytest.skip("liblopt.so not built")


@pytest.mark.parametrize("change,status", [
    (dict(param=None), BAD), (dict(state=None), BAD), (dict(n=0), BAD), (dict(n=-4), BAD), (dict(n=(1 << 38) + 1), UNSUPPORTED),
    (dict(p_dtype=3), BAD), (dict(g_dtype=-1), BAD), (dict(param=K + 2), UNSUPPORTED), (dict(grad=2 * K + 1), UNSUPPORTED),
    (dict(state=3 * K + 8), UNSUPPORTED), (dict(lr=float("nan")), BAD), (dict(lr=1e39), BAD), (dict(weight_decay=float("inf")), BAD),
    (dict(grad=K), BAD), (dict(state=K + 16), BAD), (dict(grad=3 * K + 400), BAD), (dict(param=9 * K - 8), BAD),
    (dict(state=2 * K + 3984), BAD)], ids=str)
def test_refusals_of_a_tensor(change, status):
    with pytest.raises(L.LoptError) as e:
        L.lopt_adamw_step([L.lopt_adamw_tensor(**{**TENSOR, **change})], *CALL.values())
    assert e.value.status == status, e.value
    assert len(str(e.value)) > 12


@pytest.mark.parametrize("change,status", [
    (dict(state_bits=16), BAD), (dict(beta1=1.0), BAD), (dict(beta1=-0.1), BAD), (dict(beta2=float("nan")), BAD), (dict(eps=-1e-9), BAD),
    (dict(eps=float("inf")), BAD), (dict(eps=1e39), BAD), (dict(step=None), BAD), (dict(step=9 * K + 4), UNSUPPORTED), (dict(step=3 * K + 8), BAD)], ids=str)
def test_refusals_of_the_call(change, status):
    with pytest.raises(L.LoptError) as e:
        L.lopt_adamw_step([L.lopt_adamw_tensor(**TENSOR)], *{**CALL, **change}.values())
    assert e.value.status == status, e.value


def test_tensors_that_overlap():
    """Of a long list: the same tensor twice, a state behind another's beginning; gradients may be shared."""
    def entry(k, **change):
        return L.lopt_adamw_tensor(**{**TENSOR, "param": K + k * (1 << 20), "grad": 2 * K, "state": 3 * K + k * (1 << 20), **change})
    for change in (dict(param=K + 7 * (1 << 20)), dict(state=3 * K + 7 * (1 << 20) + 4096), dict(param=3 * K + 7 * (1 << 20)), dict(grad=K)):
        with pytest.raises(L.LoptError, match="overlap"):
            L.lopt_adamw_step([entry(k) for k in range(200)] + [entry(200, **change)], *CALL.values())
    with pytest.raises(L.LoptError, match="ts is NULL"):
        L._check(L.load_library().lopt_adamw_step(None, 1, 32, 0.9, 0.999, 1e-8, 0, 9 * K, None))
    with pytest.raises(L.LoptError, match="negative"):
        L._check(L.load_library().lopt_adamw_step(None, -1, 32, 0.9, 0.999, 1e-8, 0, 9 * K, None))
    L.lopt_adamw_step([], *{**CALL, "step": None}.values())   # nothing to do


def test_sizes_of_moments():
    for n, blocks in ((1, 1), (256, 1), (257, 2), (1 << 38, 1 << 30)):
        assert L.lopt_adamw_state_bytes(n, 32) == blocks * 2048 and L.lopt_adamw_state_bytes(n, 8) == blocks * 528
    for args, status in (((0, 32), BAD), ((5, 4), BAD), (((1 << 38) + 1, 8), UNSUPPORTED)):
        with pytest.raises(L.LoptError) as e:
            L.lopt_adamw_state_bytes(*args)
        assert e.value.status == status
    assert L.load_library().lopt_adamw_state_bytes(5, 8, None) == BAD
    for args, status in (((None, 5, 8, 0, K, 2 * K, None), BAD), ((K, 5, 8, 7, K, 2 * K, None), BAD), ((K, 0, 8, 0, 2 * K, 3 * K, None), BAD),
                         ((K + 8, 5, 8, 0, 2 * K, 3 * K, None), UNSUPPORTED), ((K, 5, 8, 0, K + 64, None, None), BAD),
                         ((K, 5, 8, 0, 2 * K, 2 * K + 8, None), BAD), ((K, 5, 8, 0, 2 * K + 2, None, None), UNSUPPORTED)):
        with pytest.raises(L.LoptError) as e:
            L.lopt_adamw_moments(*args)
        assert e.value.status == status, args
    L.lopt_adamw_moments(K, 5, 8, 0, None, None, None)


def test_no_cpu_path():
    import torch
    from learned_optimizer_step_amd import layers
    x = torch.ones(4)
    for call in (lambda: layers.adamw_state(x), lambda: layers.adamw_moments(x, 4), lambda: L.AdamW([x]),
                 lambda: layers.adamw_step([x], [x], [x], torch.zeros(2, dtype=torch.int64), lr=1.0)):
        with pytest.raises(ValueError, match="GPU"):
            call()


@pytest.mark.parametrize("top", [15, 31])
def test_codes_of_the_definition(top):
    """Every code stands for a number that it alone is kept as, whatever the random bits; between two codes the bits decide."""
    codes = np.arange(top * 8 + 8, dtype=np.uint8)
    x = np.zeros((1, BLOCK))
    e = np.array([100], np.uint8)
    from adamw_cases import decode_codes
    x[0, :len(codes)] = decode_codes(codes[None], e, top)[0]
    for u in (0.0, 0.5, 1 - 2.0 ** -16):
        got, ge = encode(x, top, u)
        # the largest, 1.875, raises the block's exponent: every number is then of half the codes
        assert ge[0] == 101
    x[0, len(codes) - 1] = 0.0
    for u in (0.0, 0.5, 1 - 2.0 ** -16):
        got, ge = encode(x, top, u)
        assert ge[0] == 100 and np.array_equal(got[0, :len(codes) - 1], codes[:-1])
    mid = x.copy()
    mid[0, :len(codes) - 2] = 0.75 * x[0, :len(codes) - 2] + 0.25 * x[0, 1:len(codes) - 1]
    assert np.array_equal(encode(mid, top, 0.74)[0][0, :len(codes) - 2], codes[:-2])
    assert np.array_equal(encode(mid, top, 0.76)[0][0, :len(codes) - 2], codes[1:-1])


def test_the_definition_keeps_zero_and_loses_blocks_with_nan():
    state = np.zeros(3 * 528, np.uint8)
    g = np.zeros(700, np.float32)
    g[300] = np.nan
    g[600] = 1e-3
    _, _, new = step_moments(g, state, 8, (0.9, 0.999), 0, 1, 0)
    m, v = decode(new, 8)
    assert not m[0].any() and np.isnan(m[1]).all() and np.isnan(v[1]).all()
    assert abs(m[2, 600 - 512] / 1e-4 - 1) < 1 / 8 and (v[2] > 0).sum() == 1
